// Paged attention for few query rows per kv head: single tokens, drafts.
//
// A decode step reads every visible key and value once and does 4 G flops a
// byte-pair, so HBM bounds it: the kernel's work is to keep loads in flight.
// An item is 16 rows (TQ new tokens x the group's heads: one tensor-core tile
// of rows); a key tile is KW keys for each of the block's four warps.  A warp
// streams its keys through a ring of its own (cp.async groups), so nothing in the
// stream waits for another warp; the load cursor runs ahead of the compute
// cursor across item ends.  Blocks of 8 keys are looked up a window of 32 at a
// time, one a lane, and a window ahead of their use: a table entry costs a trip
// to L2 or HBM (0.6 to 1.5 us) that would otherwise stand before every step.
// KW is 16 keys for heads of 128 and 32 for heads of 64: 8 KB a stage, six
// stages of two blocks an SM in flight.  Scores and output are mma.sync m16n8k16
// with fp32 accumulators: at these intensities its rate is far from the bound.
// Each warp has its own running maximum and sum; the four join in shared memory
// when the item ends.  fp16 weights are 2^(s - m + 7): they keep all bits down to
// 2^-21 of the row's largest and are lost below 2^-32 (not 2^-14 and 2^-25: a long flat
// tail would go missing); m - 7 rounds to m - 8 at most, however large m is, and 2^8 is
// far inside the type's range.
//
// Measured: 64 requests of 100 to 8000 keys, 8 kv heads of 128, bf16: 1.15 GB in
// 186 us (190 as called), 6.2 TB/s, 0.91 of the measured copy rate.  Keys arrive 6 to 11 us after
// the launch, blocks end after 122 to 190 us (whole groups of SMs are slower than
// others), the join takes 5.  Three requests of up to 131k keys: 37 us.  One request
// of 1001 keys: 12.3 us, all of it latency.  (K and V by TMA boxes of 16 rows instead:
// 206 us; more blocks than are resident: 210 and up; a tenth or less of the work in a
// second, smaller wave: 187 to 190, and the three requests 5 us more.)
#include "paged.cuh"

namespace qmm {
namespace paged {
namespace {

constexpr int R = 16, kWarps = 4, NT = 32 * kWarps, ST = 3;

// log2 by which a row's weights are raised over its maximum.
template <typename E>
constexpr float kRaise = E::kF16 ? 7.f : 0.f;

template <int DP>
struct Tile {
  static constexpr int KW = 2048 / DP;               // keys of a warp's step
  static constexpr int KT = KW * kWarps;             // keys of a tile
  static constexpr uint32_t COLS = KW * 128;         // 64 columns of K or V of a step
  static constexpr uint32_t HALF = COLS * (DP / 64); // K or V of a step
  static constexpr uint32_t STAGE = 2 * HALF;
  static constexpr uint32_t RINGS = kWarps * ST * STAGE;
  // rings, joined output [2][R][DP], statistics [2][warps][R]
  static constexpr size_t SMEM = RINGS + 2 * R * DP * 4 + 2 * kWarps * R * 4;
};
static_assert(sizeof(PlanScratch<NT>) <= 2 * R * 64 * 4, "the plan's scratch lies in the output's room");

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <typename E>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (E::kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The warp's next steps of one item: lane l has looked up block l % BS of step
// l / BS (BS blocks of 8 keys a step).
struct Window {
  Block block;
  int b, kv, key0, lo, hi;  // key0: the warp's first key in the first step
  int steps;
};
template <int DP>
__device__ __forceinline__ Window next_window(const AttnArgs &a, Cursor &c, int warp, int lane) {
  using X = Tile<DP>;
  constexpr int BS = X::KW / 8;
  Window w{};
  if (c.left <= 0) return w;
  w.steps = min(min(32 / BS, c.left), c.tiles - c.at);
  w.b = c.b;
  w.kv = c.h / a.S;
  w.key0 = (c.tile0 + c.at) * X::KT + warp * X::KW;
  w.lo = c.lo;
  w.hi = c.hi;
  if (lane / BS < w.steps)
    w.block = look_up(a, c.b, w.key0 + lane / BS * X::KT + lane % BS * 8, c.lo, c.hi);
  c.left -= w.steps;
  c.at += w.steps;
  if (c.at == c.tiles && c.left > 0) cursor_next<X::KT>(a, c);
  return w;
}

template <typename E, int DP>
__global__ void __launch_bounds__(NT, 2) decode_kernel(const __grid_constant__ AttnArgs a) {
  using X = Tile<DP>;
  constexpr int KW = X::KW, KT = X::KT, NC = KW / 8, KS = DP / 16, BS = KW / 8;
  extern __shared__ __align__(1024) uint8_t smem[];
  float *obuf = reinterpret_cast<float *>(smem + X::RINGS);  // [2][R][DP]
  float *wm = obuf + 2 * R * DP, *wl = wm + kWarps * R;      // [warps][R]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  Cursor c = plan_block<NT, KT>(a, blockIdx.x, gridDim.x, *reinterpret_cast<PlanScratch<NT> *>(obuf));
  if (c.left <= 0) return;
  const uint32_t ring = smem_u32(smem) + warp * ST * X::STAGE;
  const Copier<DP> copier(a.D, X::COLS);

  Cursor ahead = c;  // where the lookups are
  Window now = next_window<DP>(a, ahead, warp, lane), then{};
  int64_t off = block_offset(a, now.block, now.kv);
  int step = 0, fill = 0;  // next step of the window, next stage to load
  auto issue = [&]() {
    if (step == now.steps) {
      now = then;
      step = 0;
      off = block_offset(a, now.block, now.kv);
    }
    if (step == 0) then = next_window<DP>(a, ahead, warp, lane);
    if (now.steps > 0) {
      const uint32_t dst = ring + fill * X::STAGE;
      const int key0 = now.key0 + step * KT;
#pragma unroll
      for (int x = 0; x < BS; ++x) {
        const int64_t o = __shfl_sync(0xffffffffu, off, step * BS + x);
        copier.copy(a, a.k, o, dst + 1024 * x, now.b, now.kv, key0 + 8 * x, now.lo, now.hi);
        copier.copy(a, a.v, o, dst + X::HALF + 1024 * x, now.b, now.kv, key0 + 8 * x, now.lo, now.hi);
      }
      ++step;
      if (++fill == ST) fill = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  const int q0 = lane >> 2, qc = (lane & 3) * 2;
  bool continues = c.at != 0, fresh = true;
  int stage = 0;
  while (c.left > 0) {
    const int n = min(c.left, c.tiles - c.at);
    const bool whole = c.at == 0 && n == c.tiles;
    // Q fragments and the two rows' key spans.
    uint32_t qf[KS][4];
    int lo[2], hi[2], deep_lo = 0, deep_hi = 0x7FFFFFFF;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      int i, head;
      const bool live = row_of(a, c.r, c.h, c.qt, q0 + 8 * x, &i, &head);
      const Span s = live ? span_of(a, c.r, i) : Span{0, 0};
      lo[x] = s.lo;
      hi[x] = s.hi;
      const uint16_t *q = static_cast<const uint16_t *>(a.q) + (static_cast<int64_t>(c.r.first) + i) * a.q_stride +
                          static_cast<int64_t>(head) * a.D;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int d = 16 * j + 8 * y + qc;
          qf[j][x + 2 * y] = live && d < a.D ? *reinterpret_cast<const uint32_t *>(q + d) : 0u;
        }
      }
      // Keys [deep_lo, deep_hi) every live row sees.
      if (live) {
        deep_lo = max(deep_lo, s.lo);
        deep_hi = min(deep_hi, s.hi);
      }
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      deep_lo = max(deep_lo, __shfl_xor_sync(0xffffffffu, deep_lo, x));
      deep_hi = min(deep_hi, __shfl_xor_sync(0xffffffffu, deep_hi, x));
    }
    float o[DP / 8][4], m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DP / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;

    // The block's first ST - 1 steps only load.
#pragma unroll 1
    for (int t = fresh ? 1 - ST : 0; t < n; ++t) {
      issue();
      if (t < 0) continue;
      asm volatile("cp.async.wait_group %0;" ::"n"(ST - 1) : "memory");
      __syncwarp();
      const uint32_t ks = ring + stage * X::STAGE, vs = ks + X::HALF;
      const int key0 = (c.tile0 + c.at + t) * KT + warp * KW;
      float s[NC][4] = {};
      {
        const int row = (lane & 7) + ((lane & 16) >> 1);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const int ch = 2 * (j & 3) + ((lane >> 3) & 1);
#pragma unroll
          for (int x = 0; x < NC / 2; ++x) {
            uint32_t b[4];
            ldmatrix4(ks + (j >> 2) * X::COLS + (16 * x + row) * 128 + ((ch ^ (row & 7)) << 4), b);
            mma16816<E>(s[2 * x], qf[j], b[0], b[1]);
            mma16816<E>(s[2 * x + 1], qf[j], b[2], b[3]);
          }
        }
      }
      const bool masked = key0 < deep_lo || deep_hi - key0 < KW;
      float top[2] = {m[0], m[1]};
#pragma unroll
      for (int x = 0; x < NC; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[x][e] *= a.scale_log2;
          if (masked) {
            const int key = key0 + 8 * x + qc + (e & 1);
            if (key < lo[e >> 1] || key >= hi[e >> 1]) s[x][e] = kNegInf;
          }
          top[e >> 1] = fmaxf(top[e >> 1], s[x][e]);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
        top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
      }
      // The weights' reference; a rounding of this difference is the same wherever m is.
      const float base[2] = {(top[0] == kNegInf ? 0.f : top[0]) - kRaise<E>,
                             (top[1] == kNegInf ? 0.f : top[1]) - kRaise<E>};
      if (__any_sync(0xffffffffu, top[0] != m[0] || top[1] != m[1])) {
        const float f0 = exp2_fast(m[0] - kRaise<E> - base[0]),
                    f1 = exp2_fast(m[1] - kRaise<E> - base[1]);
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
        m[0] = top[0];
        m[1] = top[1];
      }
#pragma unroll
      for (int x = 0; x < NC; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[x][e] = exp2_fast(s[x][e] - base[e >> 1]);
          l[e >> 1] += s[x][e];
        }
      // Weights rounded once to the element type for the product with V.
      const int vrow = lane & 15;
#pragma unroll
      for (int x = 0; x < NC / 2; ++x) {
        const uint32_t p[4] = {E::pack2(s[2 * x][0], s[2 * x][1]), E::pack2(s[2 * x][2], s[2 * x][3]),
                               E::pack2(s[2 * x + 1][0], s[2 * x + 1][1]),
                               E::pack2(s[2 * x + 1][2], s[2 * x + 1][3])};
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
          const int ch = 2 * (j & 3) + (lane >> 4);
          uint32_t b[4];
          ldmatrix4_t(vs + (j >> 2) * X::COLS + (16 * x + vrow) * 128 + ((ch ^ (vrow & 7)) << 4), b);
          mma16816<E>(o[2 * j], p, b[0], b[1]);
          mma16816<E>(o[2 * j + 1], p, b[2], b[3]);
        }
      }
      __syncwarp();
      if (++stage == ST) stage = 0;
    }
    fresh = false;

    // The four warps' statistics and outputs join.
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      m[x] -= kRaise<E>;  // what the weights are relative to
      if ((lane & 3) == 0) {
        wm[warp * R + q0 + 8 * x] = m[x];
        wl[warp * R + q0 + 8 * x] = l[x];
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float M = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * R + q0 + 8 * x]);
      const float f = exp2_fast(m[x] - (M == kNegInf ? 0.f : M));
#pragma unroll
      for (int j = 0; j < DP / 8; ++j) {
        o[j][2 * x] *= f;
        o[j][2 * x + 1] *= f;
      }
    }
    float *ob = obuf + (warp & 1) * R * DP;
    if (warp < 2) {
#pragma unroll
      for (int j = 0; j < DP / 8; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          *reinterpret_cast<float2 *>(ob + (q0 + 8 * x) * DP + 8 * j + qc) = make_float2(o[j][2 * x], o[j][2 * x + 1]);
    }
    // Eight threads a row from here on: thread tid has columns 4 (tid % 8) + 32 j.
    const int row = tid >> 3, col = (tid & 7) * 4;
    float M = kNegInf, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * R + row]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) L += exp2_fast(wm[w * R + row] - (M == kNegInf ? 0.f : M)) * wl[w * R + row];
    int i = 0, head = 0;
    const bool live = row_of(a, c.r, c.h, c.qt, row, &i, &head);
    __syncthreads();
    if (warp >= 2) {
#pragma unroll
      for (int j = 0; j < DP / 8; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float2 *p = reinterpret_cast<float2 *>(ob + (q0 + 8 * x) * DP + 8 * j + qc);
          *p = make_float2(p->x + o[j][2 * x], p->y + o[j][2 * x + 1]);
        }
    }
    __syncthreads();
    const float inv = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
    const int64_t token = static_cast<int64_t>(c.r.first) + i;
    uint16_t *out = static_cast<uint16_t *>(a.out) + token * a.out_stride + static_cast<int64_t>(head) * a.D;
    float *piece = slot_of<R, DP>(a, blockIdx.x, !continues);
    bool bad = false;
#pragma unroll
    for (int j = 0; j < DP / 32; ++j) {
      const int d = col + 32 * j;
      const float4 u = *reinterpret_cast<const float4 *>(obuf + row * DP + d);
      const float4 v = *reinterpret_cast<const float4 *>(obuf + R * DP + row * DP + d);
      const float4 y = make_float4((u.x + v.x) * inv, (u.y + v.y) * inv, (u.z + v.z) * inv, (u.w + v.w) * inv);
      if (!whole) {
        *reinterpret_cast<float4 *>(piece + row * DP + d) = y;
      } else if (live && d < a.D) {
        *reinterpret_cast<uint2 *>(out + d) = make_uint2(E::pack2(y.x, y.y), E::pack2(y.z, y.w));
        bad |= !(isfinite(y.x) && isfinite(y.y) && isfinite(y.z) && isfinite(y.w));
      }
    }
    if (col == 0) {
      if (!whole) {
        piece[R * DP + row] = M;
        piece[R * DP + R + row] = L;
      } else if (live && a.lse) {
        a.lse[token * a.Hq + head] = (M + log2f(L)) * kLn2;
      }
    }
    const unsigned votes = __ballot_sync(0xffffffffu, bad && isfinite(L));
    if (votes) {
      __syncwarp();
#pragma unroll 1
      for (int x = 0; x < 32; x += 8) {
        const int xi = __shfl_sync(0xffffffffu, i, x), xh = __shfl_sync(0xffffffffu, head, x);
        if (votes >> x & 0xFFu) row_alone<E>(a, c.b, xh, xi, 0, a.D);
      }
    }
    continues = false;
    c.left -= n;
    if (c.left > 0) cursor_next<KT>(a, c);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename E, int DP>
cudaError_t launch_t(AttnArgs a, size_t ws_bytes, cudaStream_t stream) {
  a.S = (a.G + R - 1) / R;
  a.Gs = (a.G + a.S - 1) / a.S;
  a.heads = a.Hkv * a.S;
  a.TQ = a.TH = R / a.Gs;
  // An item's queries, the join of its warps and its output, in key tiles.  Measured
  // at 0 / 3 / 6 / 10 / 20: 64 ragged requests 190 / 190 / 187 / 189 / 191 us, three of
  // up to 131k keys 44 / 42 / 39 / 38 / 38, drafts in a window 53 / 51 / 50 / 51 / 52.
  a.item_cost = 6;
  constexpr size_t smem = Tile<DP>::SMEM;
  const cudaError_t e = ensure_smem_limit<decode_kernel<E, DP>>(smem);
  if (e != cudaSuccess) return e;
  int blocks = 2 * sm_count();
  const size_t per_block = 2 * sizeof(float) * R * (DP + 2);
  blocks = static_cast<int>(std::min<size_t>(std::min(blocks, kMaxBlocks), ws_bytes / per_block));
  decode_kernel<E, DP><<<blocks, NT, smem, stream>>>(a);
  const cudaError_t le = cudaGetLastError();
  return le != cudaSuccess ? le : launch_join<E, R, DP>(a, blocks, stream);
}

template <typename E>
cudaError_t launch_e(const AttnArgs &a, size_t ws_bytes, cudaStream_t stream) {
  return a.D <= 64 ? launch_t<E, 64>(a, ws_bytes, stream) : launch_t<E, 128>(a, ws_bytes, stream);
}

}  // namespace
}  // namespace paged

cudaError_t launch_attention_decode(const paged::AttnArgs &a, int type, size_t ws_bytes, cudaStream_t stream) {
  return type == kTypeF16 ? paged::launch_e<ElemF16>(a, ws_bytes, stream)
                          : paged::launch_e<ElemBF16>(a, ws_bytes, stream);
}

}  // namespace qmm
