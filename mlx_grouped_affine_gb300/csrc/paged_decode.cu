// Paged attention for few query rows per kv head: single tokens, drafts.
//
// A decode step reads every visible key and value once and does 4 G flops a
// byte-pair, so HBM bounds it: the kernel's work is to keep loads in flight.
// An item is 16 rows (TQ new tokens x the group's heads: one tensor-core tile
// of rows), a key tile 64 keys, 16 for each of the block's four warps.  A warp
// streams its keys through a ring of its own (cp.async, 16 bytes a lane, rows
// swizzled by 16-byte chunks), so no barrier stands in the stream; the load
// cursor runs ahead of the compute cursor across item ends, and a key's page
// is looked up one step before its rows are fetched.  Scores and output are
// mma.sync m16n8k16 with fp32 accumulators: at these arithmetic intensities
// its rate is far from the bound.  Each warp has its own running maximum and
// sum; the four join in shared memory when the item ends.
#include "paged.cuh"

namespace qmm {
namespace paged {
namespace {

constexpr int R = 16, KW = 16, kWarps = 4, KT = KW * kWarps, NT = 32 * kWarps;

template <int DP>
__host__ __device__ constexpr int stages() { return DP == 128 ? 3 : 6; }
template <int DP>
__host__ __device__ constexpr uint32_t half_bytes() { return KW * DP * 2; }  // K or V of a step
template <int DP>
constexpr size_t smem_bytes() {
  return static_cast<size_t>(kWarps) * stages<DP>() * 2 * half_bytes<DP>() + 2 * R * DP * sizeof(float) +
         2 * kWarps * R * sizeof(float);
}

// 16 bytes global -> shared, or zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// The offset of the key that this lane looks up for the warp's step at the
// cursor (lanes 0-15 one key each), -1 where no row of the item sees one.
__device__ __forceinline__ int64_t lane_offset(const AttnArgs &a, const Cursor &c, int warp, int lane) {
  if (c.left <= 0) return -1;
  const int key = (c.tile0 + c.at) * KT + warp * KW + (lane & 15);
  return key >= c.lo && key < c.hi ? key_offset(a, c.b, c.h / a.S, key) : -1;
}

// One tile on; to the next item when this one ends.
__device__ __forceinline__ void cursor_step(const AttnArgs &a, Cursor &c) {
  --c.left;
  if (++c.at == c.tiles && c.left > 0) cursor_next<KT>(a, c);
}

template <typename E, int DP>
__global__ void __launch_bounds__(NT, 2) decode_kernel(AttnArgs a) {
  constexpr int ST = stages<DP>(), CH = DP / 8, KS = DP / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  float *obuf = reinterpret_cast<float *>(smem + kWarps * ST * 2 * half_bytes<DP>());  // [2][R][DP]
  float *wm = obuf + 2 * R * DP, *wl = wm + kWarps * R;                              // [warps][R]
  __shared__ PlanScratch<NT> scratch;
  griddep_launch_dependents();
  Cursor c = plan_block<NT, KT>(a, blockIdx.x, gridDim.x, scratch);
  if (c.left <= 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem) + warp * ST * 2 * half_bytes<DP>();
  const uint16_t *gk = static_cast<const uint16_t *>(a.k), *gv = static_cast<const uint16_t *>(a.v);

  Cursor ahead = c;  // where the loads are
  int64_t off = lane_offset(a, ahead, warp, lane);
  auto issue = [&](int stage) {
    if (ahead.left > 0) {
      const uint32_t dst = ring + stage * 2 * half_bytes<DP>();
#pragma unroll
      for (int i = 0; i < KW * CH / 32; ++i) {
        const int id = i * 32 + lane, row = id / CH, ch = id % CH;
        const int64_t o = __shfl_sync(0xffffffffu, off, row);
        const bool valid = o >= 0 && ch * 8 < a.D;
        const int64_t src = valid ? o + ch * 8 : 0;
        const uint32_t at = row * (DP * 2) + ((ch ^ (row & 7)) << 4);
        cp_async16(dst + at, gk + src, valid);
        cp_async16(dst + half_bytes<DP>() + at, gv + src, valid);
      }
      cursor_step(a, ahead);
      off = lane_offset(a, ahead, warp, lane);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < ST - 1; ++s) issue(s);

  const int q0 = lane >> 2, qc = (lane & 3) * 2;
  bool continues = c.at != 0;
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

    for (int t = 0; t < n; ++t) {
      issue(stage + ST - 1 >= ST ? stage - 1 : stage + ST - 1);
      cp_wait<ST - 1>();
      __syncwarp();
      const uint32_t ks = ring + stage * 2 * half_bytes<DP>(), vs = ks + half_bytes<DP>();
      const int key0 = (c.tile0 + c.at + t) * KT + warp * KW;
      float s[2][4] = {};
      {
        const int row = (lane & 7) + ((lane & 16) >> 1);
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const int ch = 2 * j + ((lane >> 3) & 1);
          uint32_t b[4];
          ldmatrix4(ks + row * (DP * 2) + ((ch ^ (row & 7)) << 4), b);
          mma16816<E>(s[0], qf[j], b[0], b[1]);
          mma16816<E>(s[1], qf[j], b[2], b[3]);
        }
      }
      const bool masked = key0 < deep_lo || key0 + KW > deep_hi;
      float top[2] = {m[0], m[1]};
#pragma unroll
      for (int x = 0; x < 2; ++x)
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
      float base[2] = {top[0] == kNegInf ? 0.f : top[0], top[1] == kNegInf ? 0.f : top[1]};
      if (__any_sync(0xffffffffu, top[0] != m[0] || top[1] != m[1])) {
        const float f0 = exp2_fast(m[0] - base[0]), f1 = exp2_fast(m[1] - base[1]);
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
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[x][e] = exp2_fast(s[x][e] - base[e >> 1]);
          l[e >> 1] += s[x][e];
        }
      // Weights rounded once to the element type for the product with V.
      const uint32_t p[4] = {E::pack2(s[0][0], s[0][1]), E::pack2(s[0][2], s[0][3]),
                             E::pack2(s[1][0], s[1][1]), E::pack2(s[1][2], s[1][3])};
      {
        const int row = lane & 15;
#pragma unroll
        for (int j = 0; j < DP / 16; ++j) {
          const int ch = 2 * j + (lane >> 4);
          uint32_t b[4];
          ldmatrix4_t(vs + row * (DP * 2) + ((ch ^ (row & 7)) << 4), b);
          mma16816<E>(o[2 * j], p, b[0], b[1]);
          mma16816<E>(o[2 * j + 1], p, b[2], b[3]);
        }
      }
      __syncwarp();
      if (++stage == ST) stage = 0;
    }

    // The four warps' statistics and outputs join.
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
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
    constexpr int LPR = DP / 4;  // lanes a row
#pragma unroll 1
    for (int x = tid; x < R * LPR; x += NT) {
      const int row = x / LPR, d = (x % LPR) * 4;
      float M = kNegInf, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * R + row]);
      const float base = M == kNegInf ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) L += exp2_fast(wm[w * R + row] - base) * wl[w * R + row];
      const float4 u = *reinterpret_cast<const float4 *>(obuf + row * DP + d);
      const float4 v = *reinterpret_cast<const float4 *>(obuf + R * DP + row * DP + d);
      const float4 y = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
      int i = 0, head = 0;
      const bool live = row_of(a, c.r, c.h, c.qt, row, &i, &head);
      bool bad = false;
      if (!whole) {
        float *w = slot_of<R, DP>(a, blockIdx.x, !continues);
        *reinterpret_cast<float4 *>(w + row * DP + d) = y;
        if (d == 0) {
          w[R * DP + row] = M;
          w[R * DP + R + row] = L;
        }
      } else if (live) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int64_t token = static_cast<int64_t>(c.r.first) + i;
        if (d < a.D) {
          uint16_t *out = static_cast<uint16_t *>(a.out) + token * a.out_stride + static_cast<int64_t>(head) * a.D + d;
          const float z[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
          *reinterpret_cast<uint2 *>(out) = make_uint2(E::pack2(z[0], z[1]), E::pack2(z[2], z[3]));
          bad = !(isfinite(z[0]) && isfinite(z[1]) && isfinite(z[2]) && isfinite(z[3]));
        }
        if (d == 0 && a.lse) a.lse[token * a.Hq + head] = (M + log2f(L)) * kLn2;
      }
      const unsigned votes = __ballot_sync(0xffffffffu, bad);
      if (votes) {
        __syncwarp();
#pragma unroll 1
        for (int first = 0; first < 32; first += LPR) {
          const int fi = __shfl_sync(0xffffffffu, i, first), fh = __shfl_sync(0xffffffffu, head, first);
          if ((votes >> first) & (LPR == 32 ? 0xFFFFFFFFu : (1u << (LPR & 31)) - 1u)) row_alone<E>(a, c.b, fh, fi);
        }
      }
    }
    continues = false;
    c.left -= n;
    if (c.left > 0) cursor_next<KT>(a, c);
  }
  cp_wait<0>();
}

template <typename E, int DP>
cudaError_t launch_t(AttnArgs a, size_t ws_bytes, cudaStream_t stream) {
  a.S = (a.G + R - 1) / R;
  a.Gs = (a.G + a.S - 1) / a.S;
  a.heads = a.Hkv * a.S;
  a.TQ = R / a.Gs;
  a.min_tiles = 2;
  constexpr size_t smem = smem_bytes<DP>();
  const cudaError_t e = ensure_smem_limit<decode_kernel<E, DP>>(smem);
  if (e != cudaSuccess) return e;
  int blocks = 2 * sm_count();
  const size_t per_block = 2 * sizeof(float) * R * (DP + 2);
  if (static_cast<size_t>(blocks) > ws_bytes / per_block) blocks = static_cast<int>(ws_bytes / per_block);
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
