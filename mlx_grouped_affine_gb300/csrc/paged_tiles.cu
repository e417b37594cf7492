// Paged attention in fp32 on the CUDA cores: fp32 elements, whose products no tensor
// form keeps, and 16-bit ones in heads of 136 to 256.  (16-bit types with heads of at
// most 128 have tensor-core kernels.)
//
// A block has items of 32 rows and walks key tiles of 64: K and V widened to
// fp32 in shared memory, a 4 x 4 patch of scores a thread (two float4 loads
// feed 16 multiply-adds), the softmax statistics of a row in the 16 lanes that
// share it, and 4 rows x DP/16 columns of output a thread in registers.  Its
// multiply-adds and the shared-memory loads that feed them bound it: five requests
// of 1 to 130 tokens, up to 2000 keys, fp32 heads of 64 take 50 us, about 12 of
// them at the fp32 units' rate; four fp32 prompts of 500 to 2048 tokens, heads of 128,
// 2.14 ms, 31 TFLOP/s, 0.39 of that rate.  Single tokens leave most of an item's rows
// empty: 64 requests of 100 to 8000 keys, groups of 4 in 32 rows, take 1.3 ms in fp32 and
// 4.4 ms in bf16 heads of 256 (one block an SM), 0.26 and 0.08 of the bytes' rate.  (Two blocks an SM; three or four: 53 to 60 us.  Tiles
// loaded ahead by cp.async: 57 against 55.5 us.)
#include "paged.cuh"

namespace qmm {
namespace paged {
namespace {

constexpr int R = 32, KT = 64, NT = 128;

template <int DP>
constexpr size_t smem_bytes() {
  return sizeof(float) * (R * (DP + 4) + KT * (DP + 4) + KT * DP + KT * (R + 4)) + sizeof(int64_t) * KT;
}

// Eight elements as fp32.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <typename E>
__device__ __forceinline__ void load8(const uint16_t *p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = E::to_f32(w[i] & 0xFFFFu);
    x[2 * i + 1] = E::to_f32(w[i] >> 16);
  }
}
template <typename E>
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) { load8(p, x); }

__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// c += (a0 b0, a1 b1): two fp32 multiply-adds an instruction.
__device__ __forceinline__ void fma_pair(float2 &c, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\t"
      "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "+f"(c.x), "+f"(c.y)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

template <typename E, int DP>
__global__ void __launch_bounds__(NT) tiles_kernel(const __grid_constant__ AttnArgs a) {
  using T = typename Elem<E>::type;
  extern __shared__ __align__(16) float smem[];
  float *Qs = smem;                    // [R][DP + 4]
  float *Ks = Qs + R * (DP + 4);       // [KT][DP + 4]
  float *Vs = Ks + KT * (DP + 4);      // [KT][DP]
  float *Ps = Vs + KT * DP;            // [KT][R + 4]
  int64_t *off = reinterpret_cast<int64_t *>(Ps + KT * (R + 4));
  __shared__ PlanScratch<NT> scratch;
  griddep_launch_dependents();
  Cursor c = plan_block<NT, KT>(a, blockIdx.x, gridDim.x, scratch);
  const int tid = threadIdx.x, rg = tid >> 4, kt = tid & 15, lane = tid & 31;
  constexpr int VEC = DP / 8, NJ = DP / 64;
  bool continues = c.at != 0;

  while (c.left > 0) {
    // A piece: the item's tiles from c.at on, as far as the block goes.
    const int n = min(c.left, c.tiles - c.at);
    const bool whole = c.at == 0 && n == c.tiles;
    __syncthreads();
    for (int x = tid; x < R * VEC; x += NT) {
      const int row = x / VEC, d = (x % VEC) * 8;
      int i, head;
      float q[8] = {};
      if (row_of(a, c.r, c.h, c.qt, row, &i, &head) && d < a.D)
        load8<E>(static_cast<const T *>(a.q) + (static_cast<int64_t>(c.r.first) + i) * a.q_stride +
                     static_cast<int64_t>(head) * a.D + d, q);
      store8(Qs + row * (DP + 4) + d, q);
    }
    Span span[4];
    float m[4], l[4];
    float2 o[4][NJ][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int t, head;
      span[i] = Span{0, 0};
      if (row_of(a, c.r, c.h, c.qt, 4 * rg + i, &t, &head)) span[i] = span_of(a, c.r, t);
      m[i] = kNegInf;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) o[i][j][e] = make_float2(0.f, 0.f);
    }
    for (int tile = c.tile0 + c.at; tile < c.tile0 + c.at + n; ++tile) {
      const int key0 = tile * KT;
      __syncthreads();
      if (tid < KT)
        off[tid] = key0 + tid >= c.lo && key0 + tid < c.hi
                       ? key_offset(a, c.b, c.h / a.S, key0 + tid) : -1;
      __syncthreads();
      for (int x = tid; x < KT * VEC; x += NT) {
        const int key = x / VEC, d = (x % VEC) * 8;
        float k[8] = {}, v[8] = {};
        if (off[key] >= 0 && d < a.D) {
          load8<E>(static_cast<const T *>(a.k) + off[key] + d, k);
          load8<E>(static_cast<const T *>(a.v) + off[key] + d, v);
        }
        store8(Ks + key * (DP + 4) + d, k);
        store8(Vs + key * DP + d, v);
      }
      __syncthreads();
      float2 s2[4][4] = {};  // sums of even and odd columns
#pragma unroll 2
      for (int d = 0; d < DP; d += 4) {
        float4 q[4], k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[i] = *reinterpret_cast<const float4 *>(Qs + (4 * rg + i) * (DP + 4) + d);
          k[i] = *reinterpret_cast<const float4 *>(Ks + (kt + 16 * i) * (DP + 4) + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            fma_pair(s2[i][j], q[i].x, q[i].y, k[j].x, k[j].y);
            fma_pair(s2[i][j], q[i].z, q[i].w, k[j].z, k[j].w);
          }
      }
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
      float4 p[4];  // the thread's four keys, four rows each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = m[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = key0 + kt + 16 * j;
          s[i][j] = key >= span[i].lo && key < span[i].hi ? s[i][j] * a.scale_log2 : kNegInf;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int x = 8; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float base = top == kNegInf ? 0.f : top;
        const float f = exp2f(m[i] - base);
        m[i] = top;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = exp2f(s[i][j] - base);
          sum += s[i][j];
          reinterpret_cast<float *>(&p[j])[i] = s[i][j];
        }
        l[i] = l[i] * f + sum;  // this lane's keys; the lanes join at the end
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) o[i][j][e] = make_float2(o[i][j][e].x * f, o[i][j][e].y * f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4 *>(Ps + (kt + 16 * j) * (R + 4) + 4 * rg) = p[j];
      __syncwarp();  // a row group's scores are written and read by the same warp
#pragma unroll 4
      for (int key = 0; key < KT; ++key) {
        const float4 w = *reinterpret_cast<const float4 *>(Ps + key * (R + 4) + 4 * rg);
        const float wi[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float4 v = *reinterpret_cast<const float4 *>(Vs + key * DP + 64 * j + 4 * kt);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            fma_pair(o[i][j][0], wi[i], wi[i], v.x, v.y);
            fma_pair(o[i][j][1], wi[i], wi[i], v.z, v.w);
          }
        }
      }
    }
    // The piece's rows: to the output, or to the workspace when the item is cut.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int x = 8; x; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
      const int row = 4 * rg + i;
      int t = 0, head = 0;
      const bool live = row_of(a, c.r, c.h, c.qt, row, &t, &head);
      bool bad = false;
      if (!whole) {
        float *w = slot_of<R, DP>(a, blockIdx.x, !continues);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          *reinterpret_cast<float4 *>(w + row * DP + 64 * j + 4 * kt) =
              make_float4(o[i][j][0].x, o[i][j][0].y, o[i][j][1].x, o[i][j][1].y);
        if (kt == 0) {
          w[R * DP + row] = m[i];
          w[R * DP + R + row] = l[i];
        }
      } else if (live) {
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        const int64_t token = static_cast<int64_t>(c.r.first) + t;
        T *out = static_cast<T *>(a.out) + token * a.out_stride + static_cast<int64_t>(head) * a.D;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = 64 * j + 4 * kt + e;
            if (d < a.D) {
              const float y = (e & 1 ? o[i][j][e >> 1].y : o[i][j][e >> 1].x) * inv;
              out[d] = Elem<E>::from_f32(y);
              bad |= !isfinite(y);
            }
          }
        if (kt == 0 && a.lse) a.lse[token * a.Hq + head] = (m[i] + log2f(l[i])) * kLn2;
      }
      // Both half-warps' rows, one after the other, by the whole warp.
      const unsigned votes = __ballot_sync(0xffffffffu, bad && isfinite(l[i]));
      if (votes) {
        __syncwarp();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int ht = __shfl_sync(0xffffffffu, t, 16 * half);
          const int hh = __shfl_sync(0xffffffffu, head, 16 * half);
          if (votes & (0xFFFFu << (16 * half))) row_alone<E>(a, c.b, hh, ht, 0, a.D);
        }
      }
    }
    c.left -= n;
    continues = false;
    if (c.left > 0) cursor_next<KT>(a, c);
  }
  (void)lane;
}

template <typename E, int DP>
cudaError_t launch_t(AttnArgs a, size_t ws_bytes, cudaStream_t stream) {
  a.S = (a.G + R - 1) / R;
  a.Gs = (a.G + a.S - 1) / a.S;
  a.heads = a.Hkv * a.S;
  a.TQ = a.TH = R / a.Gs;
  a.item_cost = 1;  // measured at 0 / 1 / 3 on the five requests above: 53 / 51 / 56 us
  constexpr size_t smem = smem_bytes<DP>();
  const cudaError_t e = ensure_smem_limit<tiles_kernel<E, DP>>(smem);
  if (e != cudaSuccess) return e;
  int blocks = sm_count() * (DP <= 128 ? 2 : 1);
  const size_t per_block = 2 * sizeof(float) * R * (DP + 2);
  blocks = static_cast<int>(std::min<size_t>(std::min(blocks, kMaxBlocks), ws_bytes / per_block));
  tiles_kernel<E, DP><<<blocks, NT, smem, stream>>>(a);
  const cudaError_t le = cudaGetLastError();
  return le != cudaSuccess ? le : launch_join<E, R, DP>(a, blocks, stream);
}

}  // namespace
}  // namespace paged

cudaError_t launch_attention_tiles(paged::AttnArgs a, int type, size_t ws_bytes, cudaStream_t stream) {
  if (type == kTypeBF16) return paged::launch_t<ElemBF16, 256>(a, ws_bytes, stream);
  if (type == kTypeF16) return paged::launch_t<ElemF16, 256>(a, ws_bytes, stream);
  if (a.D <= 64) return paged::launch_t<paged::ElemF32, 64>(a, ws_bytes, stream);
  if (a.D <= 128) return paged::launch_t<paged::ElemF32, 128>(a, ws_bytes, stream);
  return paged::launch_t<paged::ElemF32, 256>(a, ws_bytes, stream);
}

}  // namespace qmm
