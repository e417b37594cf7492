// Kernels of qmm_moe_experts and qmm_moe_layer, instantiated per code width by
// moe_bits_*.cu.
//
// With w = s c + b per group of G codes, a row's product with x over one group is
// s * sum(c x) + b * sum(x).  Codes are exact in bf16, so sum(c x) and sum(x) run on the
// tensor cores (mma.sync m16n8k16, fp32 sums) and s and b are applied to them in fp32: no
// weight is ever rounded, and s and b cost two multiply-adds per group and output instead
// of one per code.  x goes in as bf16: as it stands where it is bf16, else as a sum of two
// (fp16) or three (fp32) bf16 planes that hold it exactly, one product each.
//
// The weights that the routing asks for are streamed once; everything else (x, h, scales'
// sectors) stays in L1 or L2.  Bound by memory, then by the instructions that spread codes
// (9 per 8 codes of 4 bits).  A warp works on its own: 32 weight rows (two 16-row tiles of
// the MMA, sharing the x operand) and a range of chunks of 128 or 256 columns.  A chunk's
// codes come by TMA, a box of 16 rows per tile, into a ring of the warp's own, so that loads
// in flight cost no registers and need no block barrier.  (Copies by the lanes themselves
// touch eight rows an instruction and were held up at one cache line a cycle: 2500 cycles
// for 2048 codes a warp.)  8 slots fill the MMA's columns; 16 slots of an expert are taken
// per pass over its weights.
#pragma once
#include "moe_route.cuh"

namespace qmm {

constexpr int kMoeThreads = 256, kMoeWarps = kMoeThreads / 32;
constexpr int kMoePass = 16;      // slots of an expert per pass over its weights
constexpr int kMoeMaxCluster = 8;

template <int N>
struct Int {
  static constexpr int value = N;
};

// What the kernels share of a call.
struct MoeArgs {
  Routing route;
  ExpertWeights w;
  const uint16_t *x;    // bf16 planes [planes][tokens][hidden]
  int64_t x_plane;      // elements between planes of x
  int x_planes;
  uint16_t *h;          // silu(gate) * up: bf16 planes [h_planes][slots][inner]
  int64_t h_plane;
  int h_planes;
  int tokens;
  void *y;
  int y_type;
  unsigned *err;
  uint32_t wait_limit;
};

// ------------------------------------------------------------- the plan ----
// Which slots (token * top_k + place) go to which expert.  Every block works it out for
// itself: that is cheaper than waiting for another kernel's answer.  A unit is an expert
// with up to kMoePass of its slots; an expert's units follow one another, its slots are in
// order, and experts come in the order of their first slots, so that all blocks agree.
struct alignas(16) MoePlan {
  int units;
  int table[kMoeMaxExperts];                   // slots of an expert; then its first in `list` | first unit << 16
  short unit_expert[kMoeMaxSlots];
  short unit_first[kMoeMaxSlots];              // in `list`
  short unit_count[kMoeMaxSlots];
  short list[kMoeMaxSlots];                    // slots, unit by unit
  short slot_expert[kMoeMaxSlots];             // -1: no part in y
  short slot_place[kMoeMaxSlots];              // among its expert's slots
  float slot_weight[kMoeMaxSlots];
};

template <int NV>
__device__ __noinline__ void route_token(Routing r, int experts, int t, int lane, int *id, float *weight) {
  int i;
  float w;
  route_row<NV>(r, experts, t, lane, i, w);
  *id = i;
  *weight = w;
}

// By value: what is passed by reference would be read through memory again and again.
static __device__ __noinline__ void make_plan(const Routing r, const int tokens, const int experts, unsigned *err,
                                              MoePlan &p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, top = r.top_k;
  for (int e = threadIdx.x; e < experts; e += kMoeThreads) p.table[e] = 0;
  for (int t = warp; t < tokens; t += kMoeWarps) {
    int id = -1;
    float weight = 0.0f;
    if (!r.logits) {
      if (lane < top) id = r.ids[t * top + lane], weight = r.weights[t * top + lane];
    } else if (experts <= 128) {
      route_row<4>(r, experts, t, lane, id, weight);
    } else if (experts <= 256) {
      route_row<8>(r, experts, t, lane, id, weight);
    } else {
      route_token<32>(r, experts, t, lane, &id, &weight);
    }
    if (lane < top) {
      if (id < 0 || id >= experts) {
        if (blockIdx.x == 0) atomicOr(err, kErrIndexBit);
        id = -1;
      }
      if (weight == 0.0f) id = -1;
      p.slot_expert[t * top + lane] = static_cast<short>(id);
      p.slot_weight[t * top + lane] = weight;
    }
  }
  __syncthreads();
  const int slots = tokens * top;
  if (warp == 0) {
    for (int s0 = 0; s0 < slots; s0 += 32) {  // places: slots of the same expert before
      const int s = s0 + lane, e = s < slots ? p.slot_expert[s] : -1;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
      const int place = __popc(same & ((1u << lane) - 1u)) + (e < 0 ? 0 : p.table[e]);
      __syncwarp();
      if (e >= 0) {
        p.slot_place[s] = static_cast<short>(place);
        if (same >> lane == 1u) p.table[e] = place + 1;  // the last of them
      }
      __syncwarp();
    }
    int before = 0;  // slots | units << 16 of the experts before
    for (int s0 = 0; s0 < slots; s0 += 32) {  // units, at each expert's first slot
      const int s = s0 + lane, e = s < slots ? p.slot_expert[s] : -1;
      const int n = e >= 0 && p.slot_place[s] == 0 ? p.table[e] : 0;
      const int units = (n + kMoePass - 1) / kMoePass, own = n | units << 16;
      int sum = own;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += o;
      }
      const int at = before + sum - own, unit = at >> 16;
      __syncwarp();
      if (n > 0) p.table[e] = at;
      for (int i = 0; i < units; ++i) {
        p.unit_expert[unit + i] = static_cast<short>(e);
        p.unit_first[unit + i] = static_cast<short>((at & 0xFFFF) + i * kMoePass);
        p.unit_count[unit + i] = static_cast<short>(min(kMoePass, n - i * kMoePass));
      }
      before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) p.units = before >> 16;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < slots; s += kMoeThreads) {
    const int e = p.slot_expert[s];
    if (e >= 0) p.list[(p.table[e] & 0xFFFF) + p.slot_place[s]] = static_cast<short>(s);
  }
  __syncthreads();
}

// ------------------------------------------------------------ the codes ----

// A lane's part of a group: the G / 4 codes [t G / 4, (t + 1) G / 4) for lane 4 g + t, so
// that the four lanes of an MMA row are in one group.
template <int BITS, int G>
struct Run {
  static constexpr int kCodes = G / 4;
  static constexpr int kBits = kCodes * BITS;
  static constexpr bool kWhole = kBits % 32 == 0;  // whole words, else shifted into place
  static constexpr int words() {
    int n = 0;
    for (int t = 0; t < 4; ++t) {
      const int w = (t * kBits % 32 + kBits + 31) / 32;
      n = w > n ? w : n;
    }
    return n;
  }
  static constexpr int kWords = words();
  // Words read at once: as many as the run's alignment (its own size) allows.
  static constexpr int kPiece = !kWhole ? 1 : kWords % 4 == 0 ? 4 : kWords % 2 == 0 ? 2 : 1;
  // Codes j and j + half of a word share a register (one mask for both) where a word holds
  // whole codes; otherwise neighbours do.
  static constexpr bool kSplit = kWhole && (BITS == 2 || BITS == 4 || BITS == 8);
  static constexpr int kSub = kCodes < 16 ? kCodes : 16;  // codes spread at a time
  // A chunk: what a warp's ring holds per stage of each row, at most 128 bytes.
  static constexpr int kChunk = BITS <= 2 ? 256 : 128;
  static constexpr int kSteps = kChunk / G;
  static constexpr int kRowBytes = kChunk * BITS / 8;
  static constexpr int kStageBytes = 2 * 16 * kRowBytes;
  static constexpr int kDepth = kStageBytes >= 3072 ? 2 : kStageBytes >= 2048 ? 3 : 4;
  static constexpr CUtensorMapSwizzle kSwizzle = kRowBytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                                 : kRowBytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                                   : CU_TENSOR_MAP_SWIZZLE_NONE;
  // Place of byte `off` of a box: TMA swaps 16-byte units so that rows start in other banks.
  __device__ static __forceinline__ uint32_t place(uint32_t off) {
    if constexpr (kRowBytes == 128) return off ^ (off >> 3 & 0x70u);
    if constexpr (kRowBytes == 64) return off ^ (off >> 3 & 0x30u);
    return off;
  }
};

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Codes as bf16 pairs, each code * 2^-6.  A bf16 pattern P <= 0xFF is worth P * 2^-133, so
// a code at bit o of a half reads as c * 2^(o - 133), and times 2^(127 - o) it is exact and
// normal.  sum(x) is taken times 2^-6 too, and the sums times 2^6 at the end.
constexpr float kUnscale = 64.0f;
constexpr uint32_t kOnes = 0x3C803C80u;  // 2^-6
template <int BITS, int G>
__device__ __forceinline__ void spread_codes(const uint32_t *v, int sub, uint32_t (&p)[Run<BITS, G>::kSub / 2]) {
  using R = Run<BITS, G>;
  if constexpr (R::kSplit) {
    constexpr int kHalf = 16 / BITS, kPerSub = R::kSub * BITS / 32;
    constexpr uint32_t kMask = ((1u << BITS) - 1u) * 0x00010001u;
#pragma unroll
    for (int i = 0; i < kPerSub; ++i) {
      const uint32_t w = v[sub * kPerSub + i];
#pragma unroll
      for (int j = 0; j < kHalf; ++j) {
        const int o = j * BITS % 8, sh = j * BITS - o;
        p[i * kHalf + j] = bf16x2_mul((w >> sh) & (kMask << o), ((254u - o) << 7) * 0x00010001u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < R::kSub / 2; ++i)
      p[i] = bf16x2_mul(pair_at<BITS>(v, sub * R::kSub + 2 * i), (254u << 7) * 0x00010001u);
  }
}

// x of those codes, in the same pairs.
template <int BITS, int G>
__device__ __forceinline__ void pair_x(const uint16_t *x, uint32_t (&p)[Run<BITS, G>::kSub / 2]) {
  using R = Run<BITS, G>;
  uint32_t n[R::kSub / 2];
#pragma unroll
  for (int i = 0; i < R::kSub / 8; ++i) {
    const uint4 u = *reinterpret_cast<const uint4 *>(x + 8 * i);
    n[4 * i] = u.x, n[4 * i + 1] = u.y, n[4 * i + 2] = u.z, n[4 * i + 3] = u.w;
  }
  if constexpr (R::kSplit) {
    constexpr int kHalf = 16 / BITS;
#pragma unroll
    for (int i = 0; i < R::kSub / 2; ++i) {
      const int word = i / kHalf, j = i % kHalf, at = word * kHalf + j / 2;
      p[i] = prmt(n[at], n[at + kHalf / 2], j & 1 ? 0x7632u : 0x5410u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < R::kSub / 2; ++i) p[i] = n[i];
  }
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------- the ring ----

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t *v) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a));
}

// Scales and biases of a chunk, of the row that this lane stands for: row g + 8 (t % 2) of
// tile t / 2 for lane 4 g + t.  16-bit types are kept in pairs.
template <int STEPS>
struct Scales {
  uint32_t s[STEPS], b[STEPS];
  __device__ __forceinline__ void load(const char *ps, const char *pb, int type, int64_t at, int j0, int groups) {
    // (rows begin at multiples of `groups`, so whole chunks are aligned where it is one of STEPS)
    if (type == kTypeF32) {
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const bool in = j0 + i < groups;
        s[i] = in ? __ldg(reinterpret_cast<const uint32_t *>(ps) + at + j0 + i) : 0u;
        b[i] = in ? __ldg(reinterpret_cast<const uint32_t *>(pb) + at + j0 + i) : 0u;
      }
      return;
    }
    const uint16_t *hs = reinterpret_cast<const uint16_t *>(ps) + at + j0, *hb = reinterpret_cast<const uint16_t *>(pb) + at + j0;
    if (STEPS > 1 && groups % STEPS == 0) {
      if constexpr (STEPS == 2) {
        s[0] = __ldg(reinterpret_cast<const uint32_t *>(hs));
        b[0] = __ldg(reinterpret_cast<const uint32_t *>(hb));
      } else if constexpr (STEPS == 4) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(hs)), v = __ldg(reinterpret_cast<const uint2 *>(hb));
        s[0] = u.x, s[1] = u.y, b[0] = v.x, b[1] = v.y;
      } else if constexpr (STEPS == 8) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(hs)), v = __ldg(reinterpret_cast<const uint4 *>(hb));
        s[0] = u.x, s[1] = u.y, s[2] = u.z, s[3] = u.w;
        b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < STEPS; i += 2) {
      uint32_t h[4] = {};
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (i + k < STEPS && j0 + i + k < groups) h[k] = __ldg(hs + i + k), h[2 + k] = __ldg(hb + i + k);
      s[i / 2] = h[0] | h[1] << 16;
      b[i / 2] = h[2] | h[3] << 16;
    }
  }
};

// The MMA's columns: rows of x (or h) of up to 8 HALVES slots, lane 4 g + t reading column g.
template <int HALVES>
struct Columns {
  const uint16_t *x[HALVES];  // this lane's column of each half of the pass, at its run
  bool live[HALVES];
  int planes;
  int64_t plane;
};

// One chunk of 32 rows: acc[half][2 q + column] += s sum(c x) + b sum(x) over its groups
// from j0 on (below `groups`), q = 2 tile + row half.
template <int BITS, int G, int HALVES>
__device__ __forceinline__ void consume(uint32_t stage, int lane, const Columns<HALVES> &c, int j0, int groups,
                                        const Scales<Run<BITS, G>::kSteps> &sc, int sb_type, float (&acc)[HALVES][8]) {
  using R = Run<BITS, G>;
  const int t = lane % 4;
#pragma unroll
  for (int step = 0; step < R::kSteps; ++step) {
    if (j0 + step >= groups) break;
    float part[HALVES][2][4] = {}, ones[HALVES][4] = {};
    uint32_t v[4][R::kWords + 1];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t box = stage + (q / 2) * (16 * R::kRowBytes);
      const uint32_t at = (lane / 4 + (q % 2) * 8) * R::kRowBytes + step * (G * BITS / 8) + t * R::kBits / 32 * 4;
#pragma unroll
      for (int i = 0; i < R::kWords; i += R::kPiece) lds_words<R::kPiece>(box + R::place(at + 4 * i), &v[q][i]);
      v[q][R::kWords] = 0;
      if constexpr (!R::kWhole) {
        const uint32_t sh = t * R::kBits % 32;
#pragma unroll
        for (int i = 0; i < R::kWords; ++i) v[q][i] = __funnelshift_r(v[q][i], v[q][i + 1], sh);
      }
    }
#pragma unroll
    for (int sub = 0; sub < R::kCodes / R::kSub; ++sub) {
      uint32_t code[4][R::kSub / 2];
#pragma unroll
      for (int q = 0; q < 4; ++q) spread_codes<BITS, G>(v[q], sub, code[q]);
#pragma unroll
      for (int half = 0; half < HALVES; ++half) {
        // the smallest parts of x first
        const uint16_t *px = c.x[half] + (j0 + step) * G + sub * R::kSub + (c.planes - 1) * c.plane;
#pragma unroll 1
        for (int plane = c.planes; plane > 0; --plane, px -= c.plane) {
          uint32_t x[R::kSub / 2] = {};
          if (c.live[half]) pair_x<BITS, G>(px, x);
#pragma unroll
          for (int m = 0; m < R::kSub / 4; ++m) {
#pragma unroll
            for (int tile = 0; tile < 2; ++tile)
              mma_bf16(part[half][tile], code[2 * tile][2 * m], code[2 * tile + 1][2 * m], code[2 * tile][2 * m + 1],
                       code[2 * tile + 1][2 * m + 1], x[2 * m], x[2 * m + 1]);
            mma_bf16(ones[half], kOnes, kOnes, kOnes, kOnes, x[2 * m], x[2 * m + 1]);
          }
        }
      }
    }
    float sq[4], bq[4];
    if (sb_type == kTypeF32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sq[q] = __uint_as_float(__shfl_sync(0xFFFFFFFFu, sc.s[step], q, 4));
        bq[q] = __uint_as_float(__shfl_sync(0xFFFFFFFFu, sc.b[step], q, 4));
      }
    } else {
      const uint32_t both = prmt(sc.s[step / 2], sc.b[step / 2], step & 1 ? 0x7632u : 0x5410u);
      uint32_t u[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) u[q] = __shfl_sync(0xFFFFFFFFu, both, q, 4);
      if (sb_type == kTypeBF16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sq[q] = __uint_as_float(u[q] << 16), bq[q] = __uint_as_float(u[q] & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) sq[q] = ElemF16::to_f32(u[q] & 0xFFFFu), bq[q] = ElemF16::to_f32(u[q] >> 16);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int half = 0; half < HALVES; ++half)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float &y = acc[half][2 * q + i];
          y = fmaf(sq[q], part[half][q / 2][2 * (q % 2) + i], fmaf(bq[q], ones[half][i], y));
        }
  }
}

// Brings a chunk of x of the unit's slots into L1 ahead of its use: a 4-byte copy of each
// 32-byte sector to a place that nothing reads.
template <int CHUNK, bool TOKENS>
__device__ __forceinline__ void touch_x(uint32_t scratch, const uint16_t *x, int64_t plane, int planes, const short *slots,
                                        int count, int top, int width, int chunk, int lane) {
  constexpr int kSectors = CHUNK / 16;
  const int all = count * kSectors;
  for (int p = 0; p < planes; ++p) {
    for (int i = lane; i < all; i += 32) {
      const int slot = slots[i / kSectors], at = chunk * CHUNK + i % kSectors * 16;
      const uint16_t *from = x + p * plane + static_cast<int64_t>(TOKENS ? slot / top : slot) * width + at;
      if (at < width)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(scratch + 4 * lane), "l"(from) : "memory");
    }
  }
}

// A weight whose boxes are loaded.  Rows that are no multiple of 16 bytes long (hidden or
// inner times bits no multiple of 128, which 4 and 8 bits never are) are out of TMA's reach:
// the warp then copies its chunks itself, as it comes to them.
struct Source {
  const CUtensorMap *map;
  const uint32_t *w;  // where the warp copies, else null
  int words;          // of a row
};

// A warp's ring of chunks.
template <int BITS, int G>
struct Ring {
  using R = Run<BITS, G>;
  uint32_t base;
  uint64_t *bars;
  int lane, in, out;
  uint32_t parity;   // of the stage to read next
  int flying;        // chunks issued and not yet waited for
  bool dead;         // a wait ran out: nothing more is issued or read

  __device__ __forceinline__ void init(unsigned char *stages, uint64_t *barriers, int warp, int lane_) {
    base = smem_u32(stages) + warp * (R::kDepth * R::kStageBytes);
    bars = barriers + warp * R::kDepth;
    lane = lane_;
    in = out = flying = 0;
    parity = 0;
    dead = false;
    if (lane == 0) {
      for (int i = 0; i < R::kDepth; ++i) mbar_init(&bars[i], 1);
      asm volatile("fence.mbarrier_init.release.cluster;\n\tfence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
  }
  // Chunk `chunk` of the 16 rows at y0 of map0 and at y1 of map1.
  __device__ __forceinline__ void issue(const Source &s0, const Source &s1, int y0, int y1, int chunk) {
    const uint32_t st = base + in * R::kStageBytes;
    constexpr int kRowWords = R::kRowBytes / 4;
    if (BITS != 4 && BITS != 8 && s0.w) {
      for (int i = lane; i < 32 * kRowWords; i += 32) {
        const int row = i / kRowWords, at = i - row * kRowWords, word = chunk * kRowWords + at;
        const uint32_t *p = (row < 16 ? s0.w : s1.w) + static_cast<int64_t>((row < 16 ? y0 : y1) + row % 16) * s0.words;
        const uint32_t v = word < s0.words ? __ldg(p + word) : 0u;
        const uint32_t to = st + row / 16 * (R::kStageBytes / 2) + R::place((row % 16) * R::kRowBytes + 4 * at);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
      }
    } else if (lane == 0) {
      mbar_expect_tx(&bars[in], R::kStageBytes);
      load_box(st, s0.map, chunk * kRowWords, y0, &bars[in]);
      load_box(st + R::kStageBytes / 2, s1.map, chunk * kRowWords, y1, &bars[in]);
    }
    in = in + 1 == R::kDepth ? 0 : in + 1;
    ++flying;
  }
  // Waits for the oldest chunk; its stage, or 0 if the wait ran out.
  __device__ __forceinline__ uint32_t wait(bool copied, uint32_t limit, unsigned *err) {
    uint32_t polls = 0;
    if (BITS != 4 && BITS != 8 && copied) {
      __syncwarp();
      return base + out * R::kStageBytes;
    }
    while (!__all_sync(0xFFFFFFFFu, mbar_try_wait(&bars[out], parity))) {
      if (++polls >= limit) {
        if (lane == 0) atomicOr(err, kErrTimeoutBit);
        dead = true;
        return 0;
      }
    }
    return base + out * R::kStageBytes;
  }
  // The stage may be filled again.
  __device__ __forceinline__ void done() {
    __syncwarp();
    out = out + 1 == R::kDepth ? 0 : out + 1;
    if (out == 0) parity ^= 1;
    --flying;
  }
  // No copy may land after the block has left.
  __device__ __forceinline__ void drain(bool copied, uint32_t limit, unsigned *err) {
    while (flying > 0) {
      wait(copied, limit, err);
      done();
    }
  }
};

// The bf16 planes of v: its leading bits cut off 8 at a time (three hold all 24).  What is
// not finite stays in the first.
__device__ __forceinline__ void store_planes(uint16_t *p, int64_t plane, int planes, float v) {
  for (int i = 0; i < planes; ++i) {
    const uint32_t cut = __float_as_uint(v) & 0xFFFF0000u;
    p[i * plane] = static_cast<uint16_t>(cut >> 16);
    const bool more = (cut & 0x7F800000u) != 0x7F800000u;
    v = more ? v - __uint_as_float(cut) : 0.0f;
  }
}

// -------------------------------------------------------- gate and up ----

struct alignas(1024) GateUpShared {  // the ring follows: swizzled boxes want 1024
  MoePlan plan;
  // [0]: sums of a task that goes on in the next warp, [1]: of one that began in an earlier
  alignas(16) float sums[2][kMoeWarps][32][kMoePass];
  int task[2][kMoeWarps];  // which; -1: none
  alignas(16) uint64_t bars[kMoeWarps * 4];
  uint32_t unread[32];
};
struct MoeMaps {
  CUtensorMap gate, up, down;
};

__device__ __forceinline__ float silu_times(float gate, float up) {
  gate *= kUnscale, up *= kUnscale;
  return __fdividef(gate, 1.0f + expf(-gate)) * up;
}

// h = silu(gate x) * (up x).  A task is a unit and 16 rows of gate and of up.  A block has
// a run of tasks, whose chunks, in order, are cut evenly over its warps; a task within one
// warp is finished there (gate and up of a row are in the same lane), one that is cut is
// joined through shared memory at the end.
template <int BITS, int G>
struct GateUp {
  using R = Run<BITS, G>;
  const MoeArgs &a;
  GateUpShared &sh;
  Ring<BITS, G> ring;
  Source gate, up;
  const char *scales, *biases;
  bool copied;
  int lane, warp, tiles, groups, chunks;
  int first_unit, first_tile;        // the block's first task
  int task, chunk, unit, tile, left;  // what is multiplied next, chunks left to this warp
  int l_chunk, l_unit, l_tile, l_left;  // what is loaded next
  bool l_fresh;                       // its unit's x is not in L1 yet
  Scales<R::kSteps> next;

  __device__ __forceinline__ void advance_load() {
    if (l_left <= 0 || ring.dead) return;
    const int row = sh.plan.unit_expert[l_unit] * a.w.inner + l_tile * 16;
    ring.issue(gate, up, row, row, l_chunk);
    if (l_fresh)
      touch_x<R::kChunk, true>(smem_u32(sh.unread), a.x, a.x_plane, a.x_planes, &sh.plan.list[sh.plan.unit_first[l_unit]],
                               sh.plan.unit_count[l_unit], a.route.top_k, a.w.hidden, l_chunk, lane);
    --l_left;
    if (++l_chunk == chunks) {
      l_chunk = 0;
      l_fresh = false;
      if (++l_tile == tiles) l_tile = 0, ++l_unit, l_fresh = true;
    }
  }
  // The next chunk's scales, of the row that this lane stands for.
  __device__ __forceinline__ void load_scales(int u, int at_tile, int at_chunk) {
    const int64_t row = static_cast<int64_t>(sh.plan.unit_expert[u]) * a.w.inner + at_tile * 16 + lane / 4 + 8 * (lane % 2);
    next.load(scales, biases, a.w.sb_type, row * groups, at_chunk * R::kSteps, groups);
  }

  template <int HALVES>
  __device__ __forceinline__ void run_task() {
    const int g = lane / 4, t = lane % 4, count = sh.plan.unit_count[unit];
    const short *slots = &sh.plan.list[sh.plan.unit_first[unit]];
    Columns<HALVES> c;
    c.planes = a.x_planes;
    c.plane = a.x_plane;
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
      c.live[half] = 8 * half + g < count;
      const int token = c.live[half] ? slots[8 * half + g] / a.route.top_k : 0;
      c.x[half] = a.x + static_cast<int64_t>(token) * a.w.hidden + t * R::kCodes;
    }
    float acc[HALVES][8] = {};
    const int c0 = chunk, c1 = min(chunks, chunk + left);
    for (; chunk < c1 && !ring.dead; ++chunk) {
      const Scales<R::kSteps> sc = next;
      if (--left > 0) {
        const bool same = chunk + 1 < chunks, last = tile + 1 == tiles;
        load_scales(same || !last ? unit : unit + 1, same ? tile : last ? 0 : tile + 1, same ? chunk + 1 : 0);
      }
      const uint32_t stage = ring.wait(copied, a.wait_limit, a.err);
      if (stage) {
        consume<BITS, G, HALVES>(stage, lane, c, chunk * R::kSteps, groups, sc, a.w.sb_type, acc);
        ring.done();
        advance_load();
      }
    }
    if (c0 == 0 && c1 == chunks) {
#pragma unroll
      for (int half = 0; half < HALVES; ++half)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int place = 8 * half + 2 * t + i;
          if (place < count) {
            uint16_t *to = a.h + static_cast<int64_t>(slots[place]) * a.w.inner + tile * 16 + g;
            store_planes(to, a.h_plane, a.h_planes, silu_times(acc[half][i], acc[half][4 + i]));
            store_planes(to + 8, a.h_plane, a.h_planes, silu_times(acc[half][2 + i], acc[half][6 + i]));
          }
        }
    } else {
      const int kind = c0 == 0 ? 0 : 1;
      if (lane == 0) sh.task[kind][warp] = task;
#pragma unroll
      for (int half = 0; half < HALVES; ++half)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float2 *>(&sh.sums[kind][warp][(q / 2) * 16 + (q % 2) * 8 + g][half * 8 + 2 * t]) =
              make_float2(acc[half][2 * q], acc[half][2 * q + 1]);
    }
    chunk = 0;
    ++task;
    if (++tile == tiles) tile = 0, ++unit;
  }
};

template <int BITS, int G>
__global__ void __launch_bounds__(kMoeThreads, 2)
gate_up_kernel(const __grid_constant__ MoeArgs a, const __grid_constant__ MoeMaps maps) {
  using R = Run<BITS, G>;
  extern __shared__ __align__(1024) unsigned char raw[];
  GateUp<BITS, G> s{a, *reinterpret_cast<GateUpShared *>(raw)};
  s.warp = threadIdx.x / 32, s.lane = threadIdx.x % 32;
  s.ring.init(raw + sizeof(GateUpShared), s.sh.bars, s.warp, s.lane);
  if (threadIdx.x < 2 * kMoeWarps) s.sh.task[threadIdx.x / kMoeWarps][threadIdx.x % kMoeWarps] = -1;
  griddep_launch_dependents();
  make_plan(a.route, a.tokens, a.w.experts, a.err, s.sh.plan);
  s.tiles = a.w.inner / 16, s.groups = a.w.hidden / G, s.chunks = (a.w.hidden + R::kChunk - 1) / R::kChunk;
  const int64_t tasks = static_cast<int64_t>(s.sh.plan.units) * s.tiles;
  const int t0 = static_cast<int>(tasks * blockIdx.x / gridDim.x), t1 = static_cast<int>(tasks * (blockIdx.x + 1) / gridDim.x);
  const int64_t steps = static_cast<int64_t>(t1 - t0) * s.chunks;
  const int from = static_cast<int>(steps * s.warp / kMoeWarps);
  s.left = s.l_left = static_cast<int>(steps * (s.warp + 1) / kMoeWarps) - from;
  s.task = t0 + from / s.chunks;
  s.chunk = s.l_chunk = from % s.chunks;
  s.unit = s.l_unit = s.task / s.tiles;
  s.tile = s.l_tile = s.task % s.tiles;
  s.l_fresh = true;
  s.copied = static_cast<int64_t>(a.w.hidden) * BITS % 128 != 0;
  s.gate = Source{&maps.gate, s.copied ? a.w.w[0] : nullptr, a.w.hidden / 32 * BITS};
  s.up = Source{&maps.up, s.copied ? a.w.w[1] : nullptr, a.w.hidden / 32 * BITS};
  s.scales = static_cast<const char *>(s.lane % 4 < 2 ? a.w.scales[0] : a.w.scales[1]);
  s.biases = static_cast<const char *>(s.lane % 4 < 2 ? a.w.biases[0] : a.w.biases[1]);
  for (int i = 0; i < R::kDepth; ++i) s.advance_load();
  if (s.left > 0) s.load_scales(s.unit, s.tile, s.chunk);
  while (s.left > 0 && !s.ring.dead) {
    if (s.sh.plan.unit_count[s.unit] > 8) s.template run_task<2>();
    else s.template run_task<1>();
  }
  s.ring.drain(s.copied, a.wait_limit, a.err);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const int r = threadIdx.x % 16, place = threadIdx.x / 16;
  for (int w = 0; w < kMoeWarps; ++w) {
    const int task = s.sh.task[0][w];
    if (task < 0) continue;
    const int unit = task / s.tiles, tile = task % s.tiles;
    if (place >= s.sh.plan.unit_count[unit]) continue;
    float gate = s.sh.sums[0][w][r][place], up = s.sh.sums[0][w][16 + r][place];
    for (int v = w + 1; v < kMoeWarps; ++v)
      if (s.sh.task[1][v] == task) gate += s.sh.sums[1][v][r][place], up += s.sh.sums[1][v][16 + r][place];
    const int slot = s.sh.plan.list[s.sh.plan.unit_first[unit] + place];
    store_planes(a.h + static_cast<int64_t>(slot) * a.w.inner + tile * 16 + r, a.h_plane, a.h_planes, silu_times(gate, up));
  }
}

// ---------------------------------------------------------------- down ----

struct alignas(1024) DownShared {  // then the ring, then z: float [slots][32]
  MoePlan plan;
  alignas(16) float heads[kMoeWarps][kMoePass][32];
  alignas(16) uint64_t bars[kMoeWarps * 4];
  uint32_t unread[32];
  unsigned char unit_from[kMoeMaxSlots], unit_to[kMoeMaxSlots];
};

__device__ __forceinline__ float remote_f32(uint32_t addr, uint32_t rank) {
  uint32_t far;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(far) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// y = sum over a token's slots of weight * (down h).  A cluster takes 32 rows of every
// unit: the steps (unit, chunk), in order, are cut evenly over the cluster's warps, so a
// warp's first unit may have begun in another warp.  Sums from a unit's first chunk on go
// to z, those of a unit that began earlier to the warp's head; after the cluster's barrier
// its blocks add them up, token by token, in a fixed order.
template <int BITS, int G>
__global__ void __launch_bounds__(kMoeThreads, 2)
down_kernel(const __grid_constant__ MoeArgs a, const __grid_constant__ MoeMaps maps, int cluster) {
  using R = Run<BITS, G>;
  extern __shared__ __align__(1024) unsigned char raw[];
  DownShared &sh = *reinterpret_cast<DownShared *>(raw);
  float *z = reinterpret_cast<float *>(raw + sizeof(DownShared) + kMoeWarps * R::kDepth * R::kStageBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  Ring<BITS, G> ring;
  ring.init(raw + sizeof(DownShared), sh.bars, warp, lane);
  make_plan(a.route, a.tokens, a.w.experts, a.err, sh.plan);
  const int rank = blockIdx.x % cluster, row0 = blockIdx.x / cluster * 32;
  const int groups = a.w.inner / G, chunks = (a.w.inner + R::kChunk - 1) / R::kChunk;
  const int total = sh.plan.units * chunks;  // at most 2^22: sizes are at most 2^20
  // Warps that share the steps, none without any; warp w begins at step total * w / warps.
  const int warps = min(cluster * kMoeWarps, total), self = rank * kMoeWarps + warp;
  const int step0 = self < warps ? total * self / warps : total;
  const int step1 = self < warps ? total * (self + 1) / warps : total;
  // The warps that have a unit's first and last step: step s is in warp w where
  // total * w / warps <= s < total * (w + 1) / warps, so w = ((s + 1) * warps - 1) / total.
  for (int u = threadIdx.x; u < sh.plan.units; u += kMoeThreads) {
    sh.unit_from[u] = static_cast<unsigned char>(((u * chunks + 1) * warps - 1) / total);
    sh.unit_to[u] = static_cast<unsigned char>(((u + 1) * chunks * warps - 1) / total);
  }
  const char *const scales = static_cast<const char *>(a.w.scales[2]);
  const char *const biases = static_cast<const char *>(a.w.biases[2]);
  // this lane's row for scales: row g + 8 (t % 2) of tile t / 2
  auto scale_row = [&](int unit) {
    return static_cast<int64_t>(sh.plan.unit_expert[unit]) * a.w.hidden + row0 + g + 8 * t;
  };

  const bool copied = static_cast<int64_t>(a.w.inner) * BITS % 128 != 0;
  const Source down{&maps.down, copied ? a.w.w[2] : nullptr, a.w.inner / 32 * BITS};
  const int first_unit = step0 / chunks, first_chunk = step0 - first_unit * chunks;
  int load_step = step0, load_unit = first_unit, load_chunk = first_chunk;
  auto touch_h = [&](int unit, int chunk) {
    touch_x<R::kChunk, false>(smem_u32(sh.unread), a.h, a.h_plane, a.h_planes, &sh.plan.list[sh.plan.unit_first[unit]],
                              sh.plan.unit_count[unit], 1, a.w.inner, chunk, lane);
  };
  auto load_next = [&](bool touch) {
    if (load_step >= step1 || ring.dead) return;
    const int row = sh.plan.unit_expert[load_unit] * a.w.hidden + row0;
    ring.issue(down, down, row, row + 16, load_chunk);
    if (touch) touch_h(load_unit, load_chunk);
    ++load_step;
    if (++load_chunk == chunks) load_chunk = 0, ++load_unit;
  };
  for (int i = 0; i < R::kDepth; ++i) load_next(false);
  Scales<R::kSteps> next;
  if (step0 < step1) next.load(scales, biases, a.w.sb_type, scale_row(first_unit) * groups, first_chunk * R::kSteps, groups);
  griddep_wait();  // h is complete; the weights above do not depend on it
  for (int i = step0, u = first_unit, k = first_chunk; i < load_step; ++i) {
    touch_h(u, k);
    if (++k == chunks) k = 0, ++u;
  }

  int step = step0;
  auto run_unit = [&](auto halves, int unit, int j0) {
    constexpr int HALVES = decltype(halves)::value;
    const int j1 = min(chunks, j0 + (step1 - step));
    const int count = sh.plan.unit_count[unit];
    const short *slots = &sh.plan.list[sh.plan.unit_first[unit]];
    Columns<HALVES> c;
    c.planes = a.h_planes;
    c.plane = a.h_plane;
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
      c.live[half] = 8 * half + g < count;
      const int slot = c.live[half] ? slots[8 * half + g] : 0;
      c.x[half] = a.h + static_cast<int64_t>(slot) * a.w.inner + t * R::kCodes;
    }
    float acc[HALVES][8] = {};
    for (int j = j0; j < j1 && !ring.dead; ++j) {
      const Scales<R::kSteps> sc = next;
      ++step;
      if (step < step1) {
        const bool same = j + 1 < chunks;
        next.load(scales, biases, a.w.sb_type, scale_row(same ? unit : unit + 1) * groups, same ? (j + 1) * R::kSteps : 0,
                  groups);
      }
      const uint32_t stage = ring.wait(copied, a.wait_limit, a.err);
      if (stage) {
        consume<BITS, G, HALVES>(stage, lane, c, j * R::kSteps, groups, sc, a.w.sb_type, acc);
        ring.done();
        load_next(true);
      }
    }
#pragma unroll
    for (int half = 0; half < HALVES; ++half)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int place = half * 8 + 2 * t + i;
        if (place < count) {
          float *to = j0 == 0 ? z + slots[place] * 32 : sh.heads[warp][place];
#pragma unroll
          for (int q = 0; q < 4; ++q) to[(q / 2) * 16 + (q % 2) * 8 + g] = acc[half][2 * q + i] * kUnscale;
        }
      }
  };
  for (int unit = first_unit; step < step1 && !ring.dead; ++unit) {
    const int j0 = unit == first_unit ? first_chunk : 0;
    if (sh.plan.unit_count[unit] > 8) run_unit(Int<2>(), unit, j0);
    else run_unit(Int<1>(), unit, j0);
  }
  ring.drain(copied, a.wait_limit, a.err);
  asm volatile("cp.async.wait_all;" ::: "memory");
  cluster_barrier();

  const uint32_t z_at = smem_u32(z) + lane * 4, heads_at = smem_u32(sh.heads) + lane * 4;
  for (int token = warp * cluster + rank; token < a.tokens; token += cluster * kMoeWarps) {
    float sum = 0.0f;
#pragma unroll 4
    for (int k = 0; k < a.route.top_k; ++k) {
      const int slot = token * a.route.top_k + k, e = sh.plan.slot_expert[slot];
      if (e < 0) continue;
      const int place = sh.plan.slot_place[slot], unit = (sh.plan.table[e] >> 16) + place / kMoePass;
      const int from = sh.unit_from[unit], to = sh.unit_to[unit];
      float v = remote_f32(z_at + slot * 128, from / kMoeWarps);
      for (int w = from + 1; w <= to; ++w)
        v += remote_f32(heads_at + ((w % kMoeWarps) * kMoePass + place % kMoePass) * 128, w / kMoeWarps);
      sum = fmaf(sh.plan.slot_weight[slot], v, sum);
    }
    const int64_t at = static_cast<int64_t>(token) * a.w.hidden + row0 + lane;
    if (a.y_type == kTypeF32) static_cast<float *>(a.y)[at] = sum;
    else static_cast<uint16_t *>(a.y)[at] = a.y_type == kTypeBF16 ? ElemBF16::from_f32(sum) : ElemF16::from_f32(sum);
  }
  cluster_barrier();  // no block leaves while another reads its sums
}

// -------------------------------------------------------------- launch ----

// Boxes of 16 rows of a chunk, over all experts' rows (none where the kernels copy).
template <int BITS, int G>
cudaError_t weight_map(CUtensorMap *map, const uint32_t *w, int64_t rows, int cols) {
  using R = Run<BITS, G>;
  const uint64_t words = static_cast<uint64_t>(cols) * BITS / 32;
  if (words % 4 != 0) return cudaSuccess;
  return encode_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, w, words, rows, words * 4, R::kRowBytes / 4, 16, R::kSwizzle);
}

template <int BITS, int G>
cudaError_t launch_moe(const MoeArgs &a, cudaStream_t stream) {
  using R = Run<BITS, G>;
  const size_t ring = kMoeWarps * R::kDepth * R::kStageBytes;
  const int slots = a.tokens * a.route.top_k;
  MoeMaps maps = {};
  const int64_t inner_rows = static_cast<int64_t>(a.w.experts) * a.w.inner;
  const int64_t hidden_rows = static_cast<int64_t>(a.w.experts) * a.w.hidden;
  cudaError_t e = weight_map<BITS, G>(&maps.gate, a.w.w[0], inner_rows, a.w.hidden);
  if (e == cudaSuccess) e = weight_map<BITS, G>(&maps.up, a.w.w[1], inner_rows, a.w.hidden);
  if (e == cudaSuccess) e = weight_map<BITS, G>(&maps.down, a.w.w[2], hidden_rows, a.w.inner);
  if (e != cudaSuccess) return e;
  {
    constexpr auto kernel = gate_up_kernel<BITS, G>;
    const size_t bytes = sizeof(GateUpShared) + ring + 16;  // a run's last word may lie past its row
    e = ensure_smem_limit<kernel>(bytes);
    if (e != cudaSuccess) return e;
    const int64_t tasks = static_cast<int64_t>(slots) * (a.w.inner / 16), most = 2 * sm_count();
    kernel<<<static_cast<unsigned>(tasks < most ? tasks : most), kMoeThreads, bytes, stream>>>(a, maps);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  constexpr auto kernel = down_kernel<BITS, G>;
  const size_t bytes = sizeof(DownShared) + static_cast<size_t>(slots) * 128 + ring;
  e = ensure_smem_limit<kernel>(bytes);
  if (e != cudaSuccess) return e;
  const int tiles = a.w.hidden / 32;
  int cluster = 1;
  while (cluster < kMoeMaxCluster && tiles * cluster < sm_count()) cluster *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * cluster);
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, maps, cluster);
}

template <int BITS>
cudaError_t launch_moe_bits(const MoeArgs &a, cudaStream_t stream) {
  switch (a.w.group) {
    case 32: return launch_moe<BITS, 32>(a, stream);
    case 64: return launch_moe<BITS, 64>(a, stream);
    default: return launch_moe<BITS, 128>(a, stream);
  }
}

// moe_bits_*.cu
cudaError_t launch_moe_bits_1_2(const MoeArgs &a, cudaStream_t stream);
cudaError_t launch_moe_bits_3(const MoeArgs &a, cudaStream_t stream);
cudaError_t launch_moe_bits_4(const MoeArgs &a, cudaStream_t stream);
cudaError_t launch_moe_bits_5_6(const MoeArgs &a, cudaStream_t stream);
cudaError_t launch_moe_bits_8(const MoeArgs &a, cudaStream_t stream);

}  // namespace qmm
