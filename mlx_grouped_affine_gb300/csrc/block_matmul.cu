// qmm_block_matmul: y = A . W^T of e4m3 codes, with fp32 scales per row and 128 columns of A
// and per 128 x 128 block of W.
//
// The scales change every 128 columns, so a sum in the tensor core may be no longer than
// that: each 128-column step is one accumulator in tensor memory (four tcgen05.mma of
// kind::f8f6f4, K = 32), which the epilogue warps read, scale and add to fp32 sums in
// registers while the next step runs into a second accumulator.  Products are exact, sums
// fp32.
//
//   warp 0      loads the codes by TMA (128-byte rows, 128-byte swizzle), one lane
//   warp 1      owns tensor memory and issues the MMAs, one lane
//   the others  epilogue
//
// The issuing lane is the pace: with warp-wide waits, a commit for the ring and another for the
// epilogue, a step took it 940 cycles, the MMAs 512.  So it waits alone, and one commit a step
// tells both that the step is done.
//
// Two kernels.  `tall`: a 128 x 256 tile of y per block, an epilogue thread a row of A and
// 128 columns of one block column of W, so that a step's factor is one number a thread.
// `flat`, for few rows of A: W's rows take the MMA's 128 lanes and up to 64 rows of A its
// columns, so that nothing is padded to 128 rows; W is streamed once for each tile of A's rows.
// K is split over a cluster, whose partial sums meet in shared memory.
//
// Measured: 2048 x 14336 x 4096 in 92.5 us, 2600 TFLOP/s, bound by the 48 KB a step and SM that
// come from L2 (products alone 62 us, with loads 89) and by the stores; 1 x 4096 x 4096 in 6.2
// us (three weights in turn), of which the 16.8 MB are 2.5: launch, first tiles, cluster barrier and join.
#include "common.cuh"

namespace qmm {
namespace {

constexpr int kStep = 128;  // columns of a scale: bytes of a tile's row

struct Args {
  const float *as, *ws;
  void *y;
  int y_type;
  int M, N, steps;  // steps of 128 columns
  unsigned *err;
  uint32_t limit;
};

// ------------------------------------------------------------- PTX glue ----

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Rows of 128 bytes, K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(1) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
// fp32 accumulator, A and B e4m3 (format 0), both K-major, M = 128.
__host__ __device__ constexpr uint32_t mma_desc(int n) {
  return (1u << 4) | static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(128 >> 4) << 24;
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"(add));
}
__device__ __forceinline__ void commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Sixteen columns of this warp's 32 lanes (complete after wait_loads).
__device__ __forceinline__ void load16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void wait_loads(uint32_t (&r)[16]) {
  // (the registers pass through, so that nothing reads them earlier)
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// Two multiply-adds: (x0, x1) += (v0 f0, v1 f1).
__device__ __forceinline__ void fma2(uint64_t &x, uint32_t v0, uint32_t v1, uint64_t f) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}" : "+l"(x) : "r"(v0), "r"(v1), "l"(f));
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  return static_cast<uint64_t>(__float_as_uint(a)) | static_cast<uint64_t>(__float_as_uint(b)) << 32;
}
__device__ __forceinline__ float half_of(uint64_t v, int i) {
  return __uint_as_float(static_cast<uint32_t>(i ? v >> 32 : v));
}

// Whole-warp bounded wait; false if it ran out or another role gave up.  (Inlined: a call would
// leave the epilogue without the registers that setmaxnreg gives it.)
__device__ __forceinline__ bool wait_slow(uint64_t *b, uint32_t parity, volatile int *abort, unsigned *err, uint32_t limit) {
  uint32_t polls = 0;
  while (!__all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity))) {
    if ((++polls & 255u) == 0 || polls >= limit) {
      int stop = *abort;
      if (!stop && polls >= limit) {
        stop = *abort = 1;
        atomicOr(err, kErrTimeoutBit);
      }
      if (__any_sync(0xFFFFFFFFu, stop)) return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait(uint64_t *b, uint32_t parity, volatile int *abort, const Args &a) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity))) return true;
  return wait_slow(b, parity, abort, a.err, a.limit);
}

// The same by one thread.
__device__ __forceinline__ bool wait_alone(uint64_t *b, uint32_t parity, volatile int *abort, const Args &a) {
  if (mbar_try_wait(b, parity)) return true;
  uint32_t polls = 0;
  while (!mbar_try_wait(b, parity)) {
    if ((++polls & 255u) == 0 || polls >= a.limit) {
      if (*abort) return false;
      if (polls >= a.limit) {
        *abort = 1;
        atomicOr(a.err, kErrTimeoutBit);
        return false;
      }
    }
  }
  return true;
}

// Step k uses stage k mod STAGES and accumulator k mod 2.  done[k mod STAGES] completes when
// its MMAs have: the loader may fill the stage again, the epilogue read the accumulator.  (It
// cannot complete once more before both have seen that: step k + STAGES needs the stage
// filled, and step k + 2 the accumulator freed.)
template <int STAGES>
struct Bars {
  uint64_t full[STAGES], done[STAGES];
  uint64_t free[2];  // accumulators
  uint64_t retired;
  uint32_t tmem;
  int abort;
};

template <int STAGES>
__device__ __forceinline__ void init_bars(Bars<STAGES> &b, uint32_t epilogue_warps) {
  for (int i = 0; i < STAGES; ++i) mbar_init(&b.full[i], 1), mbar_init(&b.done[i], 1);
  for (int i = 0; i < 2; ++i) mbar_init(&b.free[i], epilogue_warps);
  mbar_init(&b.retired, 1);
  b.abort = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void alloc_tmem(uint32_t *to, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(to)), "r"(columns));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void free_tmem(uint32_t at, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}

// Loads of a block's steps into the ring, by one lane: rows at y0 of the MMA's A tile, at y1
// of its B.
template <int STAGES, int A_BYTES, int B_BYTES>
struct Loader {
  int stage = 0;
  uint32_t phase = 0, used = 0;  // used: stages loaded at least once
  __device__ __forceinline__ bool step(Bars<STAGES> &bars, const CUtensorMap *ma, const CUtensorMap *mb, uint32_t smem, int x,
                                       int y0, int y1, const Args &a) {
    if (!wait_alone(&bars.done[stage], phase ^ 1u, &bars.abort, a)) return false;
    const uint32_t at = smem + stage * (A_BYTES + B_BYTES);
    mbar_expect_tx(&bars.full[stage], A_BYTES + B_BYTES);
    tma_load_2d(at, ma, x, y0, &bars.full[stage]);
    tma_load_2d(at + A_BYTES, mb, x, y1, &bars.full[stage]);
    used |= 1u << stage;
    if (++stage == STAGES) stage = 0, phase ^= 1u;
    return true;
  }
  // No copy may land after the block has left, or after its sums have taken the ring's place:
  // waits for the last one into each stage.  Whoever stopped early: where every step fits the
  // ring the loader itself never waits, and another role's wait is the one that runs out.
  // (Otherwise these copies have landed long since: a poll a stage.)
  __device__ __forceinline__ void drain(Bars<STAGES> &bars) {
    for (int i = 0; i < STAGES; ++i) {
      if (!(used >> i & 1u)) continue;
      const uint32_t last = i < stage ? phase : phase ^ 1u;
      for (uint32_t polls = 0; polls < kDefaultWaitLimit && !mbar_try_wait(&bars.full[i], last); ++polls) {
      }
    }
  }
};

// The MMAs of a block's steps, by one lane.
template <int STAGES, int A_BYTES, int B_BYTES, int COLUMNS>
struct Multiplier {
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  __device__ __forceinline__ bool step(Bars<STAGES> &bars, uint32_t smem, uint32_t tmem, const Args &a) {
    if (!wait_alone(&bars.free[acc], acc_phase ^ 1u, &bars.abort, a) ||
        !wait_alone(&bars.full[stage], phase, &bars.abort, a))
      return false;
    fence_after();
    const uint32_t at = smem + stage * (A_BYTES + B_BYTES);
    const uint64_t da = tile_desc(at), db = tile_desc(at + A_BYTES);
#pragma unroll
    for (int j = 0; j < kStep / 32; ++j)
      mma_e4m3(tmem + acc * COLUMNS, da + 2 * j, db + 2 * j, mma_desc(COLUMNS), j ? 1u : 0u);
    commit(&bars.done[stage]);
    if (++stage == STAGES) stage = 0, phase ^= 1u;
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
    return true;
  }
  // Every MMA issued retires before tensor memory is freed.
  __device__ __forceinline__ void retire(Bars<STAGES> &bars, uint32_t limit) {
    commit(&bars.retired);
    for (uint32_t polls = 0; polls < limit && !mbar_try_wait(&bars.retired, 0); ++polls) {
    }
  }
};

__device__ __forceinline__ void store_one(const Args &a, int64_t at, float v) {
  if (a.y_type == kTypeF32) static_cast<float *>(a.y)[at] = v;
  else static_cast<uint16_t *>(a.y)[at] = a.y_type == kTypeBF16 ? ElemBF16::from_f32(v) : ElemF16::from_f32(v);
}

// ----------------------------------------------------------------- tall ----

constexpr int kTallM = 128, kTallN = 256, kTallStages = 4;
// Three warpgroups: one loads and multiplies (two of its warps), two are the epilogue, each
// thread with 128 sums and two batches of 16 columns on their way in (tcgen05.wait::ld waits
// for every load, so one batch flies while the other is added).  384 threads start with 168
// registers; the epilogue takes what the first group gives back: 56 + 2 * 224 = 3 * 168.  (A
// spill there costs half of the rate.)
constexpr int kTallEpilogue = 8, kTallColumns = 128, kTallBatch = 16, kTallThreads = 384;
constexpr int kTallA = kTallM * kStep, kTallB = kTallN * kStep;

// Scales of four steps, fetched four steps ahead: a thread's row of A is a line of its own,
// and a load of 4 bytes a step, 32 lines a warp, held the epilogue up.
struct Factors {
  float a[4] = {}, w[4] = {};
  __device__ __forceinline__ void load(const float *as, const float *ws, int k, int steps) {
    if (steps % 4 == 0) {  // (then rows are 16-byte aligned)
      if (k >= steps) return;
      const float4 u = __ldg(reinterpret_cast<const float4 *>(as + k)), v = __ldg(reinterpret_cast<const float4 *>(ws + k));
      a[0] = u.x, a[1] = u.y, a[2] = u.z, a[3] = u.w;
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k + i < steps) a[i] = __ldg(as + k + i), w[i] = __ldg(ws + k + i);
    }
  }
};

// 64 bytes of a row of y: 16 sums (fp32) or 32.
__device__ __forceinline__ void as_output(const uint64_t *sum, int type, uint32_t (&w)[16]) {
  if (type == kTypeF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[2 * i] = static_cast<uint32_t>(sum[i]), w[2 * i + 1] = static_cast<uint32_t>(sum[i] >> 32);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float lo = half_of(sum[i], 0), hi = half_of(sum[i], 1);
      w[i] = type == kTypeBF16 ? ElemBF16::pack2(lo, hi) : ElemF16::pack2(lo, hi);
    }
  }
}

// A warp's 32 rows of 128 columns to y by TMA, 64 bytes of each row at a time, from two
// buffers of 2 KB of its own: the warp goes on while they are written.  (Stored by the threads
// themselves, each to a row of its own, they held the next tile's steps up by a quarter of the
// time of a tile.)
__device__ __forceinline__ void send_rows(const Args &a, const CUtensorMap *my, uint32_t out, int m, int n, int lane,
                                          const uint64_t (&sum)[kTallColumns / 2]) {
  auto send = [&](const uint64_t *part, int at, int buffer) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");  // the buffer's last one is read
    __syncwarp();
    uint32_t w[16];
    as_output(part, a.y_type, w);
    const uint32_t to = out + buffer * 2048 + lane * 64;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // (the 64-byte swizzle of the map)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((i ^ (lane >> 1 & 3)) << 4)), "r"(w[4 * i]),
                   "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                   : "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      if (n + at < a.N)
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(my), "r"(n + at),
                     "r"(m), "r"(out + buffer * 2048)
                     : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  };
  if (a.y_type == kTypeF32) {
#pragma unroll
    for (int r = 0; r < 8; ++r) send(&sum[8 * r], 16 * r, r % 2);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) send(&sum[16 * r], 32 * r, r % 2);
  }
}

__global__ void __launch_bounds__(kTallThreads, 1)
tall_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw,
            const __grid_constant__ CUtensorMap my, const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) unsigned char raw[];
  __shared__ Bars<kTallStages> bars;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t smem = (smem_u32(raw) + 1023u) & ~1023u;
  if (threadIdx.x == 0) {
    init_bars(bars, kTallEpilogue);
    asm volatile("prefetch.tensormap [%0];" ::"l"(&ma) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mw) : "memory");
  }
  if (warp == 1) alloc_tmem(&bars.tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars.tmem;
  const int m_tiles = (a.M + kTallM - 1) / kTallM, n_tiles = (a.N + kTallN - 1) / kTallN;
  const int64_t tiles = static_cast<int64_t>(m_tiles) * n_tiles;

  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // Lanes 32 (warp % 4) .. of tensor memory are this warp's, and a part of the columns.
    const int row = 32 * (warp % 4) + lane, first = (warp - 4) / 4 * kTallColumns;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp % 4)) << 16) + first;
    int acc = 0, stage = 0;
    uint32_t phase = 0;
    const uint32_t out = smem + kTallStages * (kTallA + kTallB) + (warp - 4) * 4096;
    const bool by_tma = a.N * (a.y_type == kTypeF32 ? 4ll : 2ll) % 16 == 0;  // rows that TMA can address
    bool ok = true;
    const float *as, *ws;
    Factors next;
    auto begin = [&](int64_t tile) {
      const int64_t m = tile % m_tiles * kTallM + row, n = tile / m_tiles * kTallN + first;
      as = a.as + (m < a.M ? m : a.M - 1) * a.steps;
      ws = a.ws + (n < a.N ? n / 128 : 0) * a.steps;
      next.load(as, ws, 0, a.steps);
    };
    begin(blockIdx.x);
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const int64_t m = tile % m_tiles * kTallM + row, n = tile / m_tiles * kTallN + first;
      uint64_t sum[kTallColumns / 2];
#pragma unroll
      for (int i = 0; i < kTallColumns / 2; ++i) sum[i] = 0;
      float four[4] = {};
      for (int k = 0; k < a.steps; ++k) {
        if (k % 4 == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) four[i] = next.a[i] * next.w[i];
          next.load(as, ws, k + 4, a.steps);
        }
        const uint64_t ff = pair(four[0], four[0]);
#pragma unroll
        for (int i = 0; i < 3; ++i) four[i] = four[i + 1];
        if (!wait(&bars.done[stage], phase, &bars.abort, a)) {
          ok = false;
          break;
        }
        fence_after();
        uint32_t v[2][kTallBatch];
        load16(at + acc * kTallN, v[0]);
#pragma unroll
        for (int c = 0; c < kTallColumns / kTallBatch; ++c) {
          wait_loads(v[c % 2]);
          if (c + 1 < kTallColumns / kTallBatch) load16(at + acc * kTallN + kTallBatch * (c + 1), v[(c + 1) % 2]);
          if (c + 1 == kTallColumns / kTallBatch) {
            fence_before();
            if (lane == 0) mbar_arrive(&bars.free[acc]);
          }
#pragma unroll
          for (int i = 0; i < kTallBatch / 2; ++i)
            fma2(sum[kTallBatch / 2 * c + i], v[c % 2][2 * i], v[c % 2][2 * i + 1], ff);
        }
        acc ^= 1;
        if (++stage == kTallStages) stage = 0, phase ^= 1u;
      }
      if (!ok) break;
      if (tile + gridDim.x < tiles) begin(tile + gridDim.x);
      if (by_tma) {
        if (m - lane < a.M) send_rows(a, &my, out, static_cast<int>(m) - lane, static_cast<int>(n), lane, sum);
      } else if (m < a.M) {
#pragma unroll
        for (int i = 0; i < kTallColumns; ++i)
          if (n + i < a.N) store_one(a, m * a.N + n + i, half_of(sum[i / 2], i % 2));
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the block's memory goes
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0 && lane == 0) {
      Loader<kTallStages, kTallA, kTallB> load;
      bool ok = true;
      for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const int m0 = static_cast<int>(tile % m_tiles) * kTallM, n0 = static_cast<int>(tile / m_tiles) * kTallN;
        for (int k = 0; ok && k < a.steps; ++k) ok = load.step(bars, &ma, &mw, smem, k * kStep, m0, n0, a);
      }
      load.drain(bars);
    } else if (warp == 1 && lane == 0) {
      Multiplier<kTallStages, kTallA, kTallB, kTallN> mul;
      bool ok = true;
      for (int64_t tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x)
        for (int k = 0; ok && k < a.steps; ++k) ok = mul.step(bars, smem, tmem, a);
      mul.retire(bars, kDefaultWaitLimit);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    free_tmem(tmem, 512);
  }
}

// ----------------------------------------------------------------- flat ----

constexpr int kFlatThreads = 192, kFlatEpilogue = 128;
template <int T>
__host__ __device__ constexpr int flat_stages() { return T <= 32 ? 5 : 4; }
template <int T>
__host__ __device__ constexpr uint32_t flat_columns() { return T == 16 ? 32 : 2 * T; }

// 128 rows of W and T rows of A; the cluster's blocks (blockIdx.x % split) share the steps.
template <int T>
__global__ void __launch_bounds__(kFlatThreads, 2)
flat_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw, const __grid_constant__ Args a,
            int split) {
  constexpr int kStages = flat_stages<T>(), kA = 128 * kStep, kB = T * kStep;
  extern __shared__ __align__(1024) unsigned char raw[];
  __shared__ Bars<kStages> bars;
  __shared__ __align__(16) float factors[2][T];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t smem = (smem_u32(raw) + 1023u) & ~1023u;
  const int rank = blockIdx.x % split, n0 = blockIdx.x / split * 128, m0 = blockIdx.y * T;
  const int k0 = static_cast<int>(static_cast<int64_t>(a.steps) * rank / split);
  const int k1 = static_cast<int>(static_cast<int64_t>(a.steps) * (rank + 1) / split);
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mw) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&ma) : "memory");
    init_bars(bars, kFlatEpilogue / 32);
  }
  if (warp == 1) alloc_tmem(&bars.tmem, flat_columns<T>());
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = bars.tmem;
  // Partial sums take the ring's place once every product has read it: [T][128].
  const uint32_t partial = smem;
  uint64_t sum[T / 2];
#pragma unroll
  for (int i = 0; i < T / 2; ++i) sum[i] = 0;
  const int row = 32 * (warp % 4) + lane;

  if (warp == 0) {
    if (lane == 0) {
      Loader<kStages, kA, kB> load;
      bool ok = true;
      for (int k = k0; ok && k < k1; ++k) ok = load.step(bars, &mw, &ma, smem, k * kStep, n0, m0, a);
      load.drain(bars);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      Multiplier<kStages, kA, kB, T> mul;
      bool ok = true;
      for (int k = k0; ok && k < k1; ++k) ok = mul.step(bars, smem, tmem, a);
      mul.retire(bars, kDefaultWaitLimit);
    }
  } else {
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp % 4)) << 16);
    const float *ws = a.ws + static_cast<int64_t>(n0 / 128) * a.steps;
    const int column = threadIdx.x - 64;  // of A's rows, whose factor this thread fetches
    const int64_t m = m0 + column;
    const float *as = a.as + (m < a.M ? m : a.M - 1) * a.steps;
    int acc = 0, stage = 0;
    uint32_t phase = 0;
    float f = column < T && k0 < k1 ? __ldg(as + k0) * __ldg(ws + k0) : 0.0f;
    bool ok = true;
    for (int k = k0; k < k1; ++k) {  // (the barrier is met by every warp, stopped early or not)
      if (column < T) factors[k % 2][column] = f;
      if (column < T && k + 1 < k1) f = __ldg(as + k + 1) * __ldg(ws + k + 1);
      asm volatile("bar.sync 1, %0;" ::"n"(kFlatEpilogue) : "memory");
      ok = ok && wait(&bars.done[stage], phase, &bars.abort, a);
      if (!ok) continue;
      fence_after();
#pragma unroll
      for (int c = 0; c < T / 16; ++c) {
        uint32_t v[16];
        load16(at + acc * T + 16 * c, v);
        wait_loads(v);
        if (c == T / 16 - 1) {
          fence_before();
          if (lane == 0) mbar_arrive(&bars.free[acc]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(&factors[k % 2][16 * c + 4 * i]);
          fma2(sum[8 * c + 2 * i], v[4 * i], v[4 * i + 1], ff.x);
          fma2(sum[8 * c + 2 * i + 1], v[4 * i + 2], v[4 * i + 3], ff.y);
        }
      }
      acc ^= 1;
      if (++stage == kStages) stage = 0, phase ^= 1u;
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 1) {
    fence_after();
    free_tmem(tmem, flat_columns<T>());
  }
  if (warp >= 2) {
#pragma unroll
    for (int c = 0; c < T; ++c)
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(partial + (c * 128 + row) * 4), "f"(half_of(sum[c / 2], c % 2)) : "memory");
  }
  cluster_barrier();
  if (warp >= 2 && n0 + row < a.N) {
    for (int c = rank; c < T && m0 + c < a.M; c += split) {
      float v = 0.0f;
#pragma unroll 4
      for (int r = 0; r < split; ++r) v += remote_f32(partial + (c * 128 + row) * 4, r);
      store_one(a, static_cast<int64_t>(m0 + c) * a.N + n0 + row, v);
    }
  }
  cluster_barrier();  // no block leaves while another reads its sums
}

// --------------------------------------------------------------- launch ----

cudaError_t code_map(CUtensorMap *map, const uint8_t *p, int rows, int cols, int box_rows) {
  return encode_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, cols, rows, cols, kStep, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows of A and blocks that share the steps in `flat`; no split: the call goes to `tall`.
//
// Two blocks fit an SM; more blocks than that are a second round, which costs more than a split
// gains (384 blocks of an eighth of the steps 28 us, 192 of a half 20.5).  So rows are halved while
// four-fold splits still fit (eight-fold from 32 steps on: 128 x 1024 x 14336 12 us against 15.5,
// 77 x 1021 x 4208 7.7 against 8.7), and then K is split for as long as blocks fit.  The cluster's blocks
// add up the rows of their tile in turns, 0.22 us a row, which few steps do not pay for: `tall`
// takes 3 us and 0.4 a step whatever its rows.  Measured, us (`flat` as chosen here / `tall`; K is
// 32 steps but where it is given):
//   M            16           32           64           128          256
//   N 1024       6.2 / 16.6   6.5 / 16.6   7.3 / 16.7   8.2 / 17.1  10.3 / 17.2
//   N 4096       8.5 / 17.0   9.5 / 17.1  11.4 / 17.2  13.2 / 17.6  21.1 / 17.7 (32 rows a block)
//   N 14336     16.2 / 18.7  18.5 / 18.5  23.2 / 18.7  29.7 / 19.3
//   N 128256    97.0 / 97.7   108 / 92
//   K 256, N 4096    5.7 / 4.5 (8 rows), M = 1: 3.9 / 4.5
//   K 512, N 4096    4.7 / 5.4   5.4 / 5.4   6.5 / 5.5 (8 rows)   8.8 / 6.2 (16)
//   K 1024, N 4096   6.4 / 7.5   6.4 / 7.6   7.5 / 7.8 (8 rows)   9.8 / 8.2 (16)
//   K 2048, N 14336  11.9 / 11.9 (8 rows)   14.2 / 11.9 (16)
//   K 8192, N 4096  11.2 / 29.7  12.2 / 29.7  13.9 / 29.7  17.2 / 30.1
struct FlatShape {
  int rows, split;
};
FlatShape flat_shape(int M, int N, int steps) {
  const int64_t n_tiles = (N + 127) / 128, room = 2 * sm_count();
  auto blocks = [&](int rows) { return n_tiles * ((M + rows - 1) / rows); };
  int rows = M <= 16 ? 16 : M <= 32 ? 32 : 64, split = 1;
  const int ways = steps < 4 ? steps : steps < 32 ? 4 : 8;
  while (rows > 16 && blocks(rows / 2) * ways <= room) rows /= 2;
  while (split < 8 && 2 * split <= steps && 2 * split * blocks(rows) <= room) split *= 2;
  const int joined = ((M < rows ? M : rows) + split - 1) / split;
  const int pays = steps < 8 ? 4 : steps < 32 ? steps / 2 : 16;
  return {rows, joined <= pays ? split : 0};
}

template <int T>
cudaError_t launch_flat(const uint8_t *pa, const uint8_t *w, int K, const Args &a, int split, cudaStream_t stream) {
  CUtensorMap ma, mw;
  cudaError_t e = code_map(&ma, pa, a.M, K, T);
  if (e == cudaSuccess) e = code_map(&mw, w, a.N, K, 128);
  if (e != cudaSuccess) return e;
  constexpr auto kernel = flat_kernel<T>;
  const size_t bytes = 1024 + static_cast<size_t>(flat_stages<T>()) * (128 + T) * kStep;
  e = ensure_smem_limit<kernel>(bytes);
  if (e != cudaSuccess) return e;
  const int n_tiles = (a.N + 127) / 128, m_tiles = (a.M + T - 1) / T;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_tiles * split, m_tiles);
  cfg.blockDim = dim3(kFlatThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mw, a, split);
}

}  // namespace

cudaError_t launch_block_matmul(const uint8_t *pa, const float *a_scales, int M, const uint8_t *w,
                                const float *w_scales, int N, int K, void *y, int y_type,
                                cudaStream_t stream) {
  Args a;
  a.as = a_scales;
  a.ws = w_scales;
  a.y = y;
  a.y_type = y_type;
  a.M = M;
  a.N = N;
  a.steps = (K + kStep - 1) / kStep;
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidSymbol;
  a.limit = wait_limit();
  const FlatShape flat = flat_shape(M, N, a.steps);
  if (flat.split > 0) {
    switch (flat.rows) {
      case 16: return launch_flat<16>(pa, w, K, a, flat.split, stream);
      case 32: return launch_flat<32>(pa, w, K, a, flat.split, stream);
      default: return launch_flat<64>(pa, w, K, a, flat.split, stream);
    }
  }
  CUtensorMap ma, mw;
  cudaError_t e = code_map(&ma, pa, M, K, kTallM);
  if (e == cudaSuccess) e = code_map(&mw, w, N, K, kTallN);
  if (e != cudaSuccess) return e;
  // y in boxes of 64 bytes by 32 rows (unused where its rows are no multiple of 16 bytes).
  CUtensorMap my = {};
  const uint64_t size = y_type == kTypeF32 ? 4 : 2;
  if (N * size % 16 == 0)
    e = encode_map_2d(&my, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, y, N, M, N * size,
                      static_cast<uint32_t>(64 / size), 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (e != cudaSuccess) return e;
  const size_t bytes = 1024 + static_cast<size_t>(kTallStages) * (kTallA + kTallB) + kTallEpilogue * 4096;
  e = ensure_smem_limit<tall_kernel>(bytes);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((M + kTallM - 1) / kTallM) * ((N + kTallN - 1) / kTallN);
  const unsigned grid = static_cast<unsigned>(tiles < sm_count() ? tiles : sm_count());
  tall_kernel<<<grid, kTallThreads, bytes, stream>>>(ma, mw, my, a);
  return cudaGetLastError();
}

}  // namespace qmm
