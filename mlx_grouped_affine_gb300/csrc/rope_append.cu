// Rotary positions on q and k, and K and V into the paged cache, in one pass.
//
// Pair i of a head (x1, x2) turns by the angle of position pos[axis(i)] and
// frequency i: (x1 c - x2 s, x2 c + x1 s), c and s from the caller's fp32
// table, products and sums in fp32, one rounding to the element type.  The
// pairs are (i, i + r/2) or (2i, 2i + 1); axis(i) follows from the sections.
//
// Nothing is read twice but the table's row, so bytes bound it: q, k, v read
// once, q, K, V written once, 16 bytes a lane.  A thread has eight pairs of a
// token for HPT heads: their cosines and sines stay in registers.
#include "paged.cuh"

namespace qmm {
namespace {

using paged::Elem;

constexpr int kMaxAxes = 4;

struct RopeArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, out_stride;
  const int *positions, *slots;
  const float *table;  // [max_pos][r]: r/2 cosines, then r/2 sines
  void *q_out, *k_cache, *v_cache;
  int64_t page_stride, head_stride, token_stride;
  unsigned *err;
  int64_t pool;        // slots of the cache
  int T, Hq, Hk, D, r, page, max_pos, axes;
  int end[kMaxAxes];   // one past each axis's last pair
};

template <typename E>
struct Vec8;  // eight elements in their own type
template <typename E>
struct Vec8 {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(uint16_t *p) const { *reinterpret_cast<uint4 *>(p) = w; }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = E::to_f32(u[i] & 0xFFFFu);
      x[2 * i + 1] = E::to_f32(u[i] >> 16);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    w = make_uint4(E::pack2(x[0], x[1]), E::pack2(x[2], x[3]), E::pack2(x[4], x[5]), E::pack2(x[6], x[7]));
  }
};
template <>
struct Vec8<paged::ElemF32> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void store(float *p) const {
    *reinterpret_cast<float4 *>(p) = a;
    *reinterpret_cast<float4 *>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Where a token's K and V go: the element offset of its head 0, or -1.
__device__ __forceinline__ int64_t slot_offset(const RopeArgs &a, int t) {
  const int slot = __ldg(a.slots + t);
  if (slot < 0) return -1;  // a token that is not kept
  if (slot >= a.pool) {
    atomicOr(a.err, kErrIndexBit);
    return -1;
  }
  const int pg = slot / a.page;
  return pg * a.page_stride + (slot - pg * a.page) * a.token_stride;
}

template <typename E, int HPT, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rope_append_kernel(RopeArgs a, int tokens_per_block, int units) {
  using T = typename Elem<E>::type;
  const int half = a.r / 2;
  const int turns = a.r / 16, keeps = (a.D - a.r) / 8, copies = a.D / 8;
  const int groups = (a.Hq + a.Hk + HPT - 1) / HPT;
  const int t0 = blockIdx.x * tokens_per_block;
  const int here = min(tokens_per_block, a.T - t0);
  for (int x = threadIdx.x; x < here * units; x += blockDim.x) {
    const int t = t0 + x / units;
    int u = x % units;
    const int64_t row = t;
    if (u < groups * turns) {
      // Eight pairs of HPT heads of q or k.
      const int h0 = u / turns * HPT, i0 = u % turns * 8;
      Vec8<E> lo[HPT], hi[HPT];
#pragma unroll
      for (int j = 0; j < HPT; ++j) {
        const int h = h0 + j;
        if (h >= a.Hq + a.Hk) continue;
        const T *p = h < a.Hq ? static_cast<const T *>(a.q) + row * a.q_stride + static_cast<int64_t>(h) * a.D
                              : static_cast<const T *>(a.k) + row * a.k_stride + static_cast<int64_t>(h - a.Hq) * a.D;
        lo[j].load(p + (INTERLEAVED ? 2 * i0 : i0));
        hi[j].load(p + (INTERLEAVED ? 2 * i0 + 8 : half + i0));
      }
      float c[8], s[8];
      bool known = true;
      int axis = 0;
      while (axis < a.axes - 1 && i0 >= a.end[axis]) ++axis;
      if (axis == a.axes - 1 || i0 + 8 <= a.end[axis]) {
        // The eight pairs share an axis.
        const int pos = __ldg(a.positions + static_cast<int64_t>(axis) * a.T + t);
        known = static_cast<unsigned>(pos) < static_cast<unsigned>(a.max_pos);
        const float *p = a.table + static_cast<int64_t>(known ? pos : 0) * a.r + i0;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 cv = __ldg(reinterpret_cast<const float4 *>(p + e));
          const float4 sv = __ldg(reinterpret_cast<const float4 *>(p + half + e));
          c[e] = cv.x; c[e + 1] = cv.y; c[e + 2] = cv.z; c[e + 3] = cv.w;
          s[e] = sv.x; s[e + 1] = sv.y; s[e + 2] = sv.z; s[e + 3] = sv.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          while (axis < a.axes - 1 && i0 + e >= a.end[axis]) ++axis;
          const int pos = __ldg(a.positions + static_cast<int64_t>(axis) * a.T + t);
          const bool ok = static_cast<unsigned>(pos) < static_cast<unsigned>(a.max_pos);
          known &= ok;
          const float *p = a.table + static_cast<int64_t>(ok ? pos : 0) * a.r + i0 + e;
          c[e] = __ldg(p);
          s[e] = __ldg(p + half);
        }
      }
      if (!known) {
        atomicOr(a.err, kErrIndexBit);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = s[e] = 0.f;
      }
      const int64_t slot = h0 + HPT > a.Hq ? slot_offset(a, t) : -1;
#pragma unroll
      for (int j = 0; j < HPT; ++j) {
        const int h = h0 + j;
        if (h >= a.Hq + a.Hk) continue;
        float x0[8], x1[8];
        lo[j].get(x0);
        hi[j].get(x1);
        if (INTERLEAVED) {
          // pairs (x[2e], x[2e + 1]) of the sixteen consecutive elements
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u0 = x0[2 * e], u1 = x0[2 * e + 1], w0 = x1[2 * e], w1 = x1[2 * e + 1];
            x0[2 * e] = u0 * c[e] - u1 * s[e];
            x0[2 * e + 1] = u1 * c[e] + u0 * s[e];
            x1[2 * e] = w0 * c[4 + e] - w1 * s[4 + e];
            x1[2 * e + 1] = w1 * c[4 + e] + w0 * s[4 + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u0 = x0[e], u1 = x1[e];
            x0[e] = u0 * c[e] - u1 * s[e];
            x1[e] = u1 * c[e] + u0 * s[e];
          }
        }
        if (!known) {  // a zero row, whatever q and k hold
#pragma unroll
          for (int e = 0; e < 8; ++e) x0[e] = x1[e] = 0.f;
        }
        lo[j].set(x0);
        hi[j].set(x1);
        T *p;
        if (h < a.Hq) {
          p = static_cast<T *>(a.q_out) + row * a.out_stride + static_cast<int64_t>(h) * a.D;
        } else {
          if (slot < 0) continue;
          p = static_cast<T *>(a.k_cache) + slot + (h - a.Hq) * a.head_stride;
        }
        lo[j].store(p + (INTERLEAVED ? 2 * i0 : i0));
        hi[j].store(p + (INTERLEAVED ? 2 * i0 + 8 : half + i0));
      }
      continue;
    }
    u -= groups * turns;
    if (u < groups * keeps) {
      // Eight elements past the rotated ones, of HPT heads of q or k.
      const int h0 = u / keeps * HPT, d = a.r + u % keeps * 8;
      Vec8<E> w[HPT];
#pragma unroll
      for (int j = 0; j < HPT; ++j) {
        const int h = h0 + j;
        if (h >= a.Hq + a.Hk) continue;
        w[j].load(h < a.Hq ? static_cast<const T *>(a.q) + row * a.q_stride + static_cast<int64_t>(h) * a.D + d
                           : static_cast<const T *>(a.k) + row * a.k_stride + static_cast<int64_t>(h - a.Hq) * a.D + d);
      }
      const int64_t slot = h0 + HPT > a.Hq ? slot_offset(a, t) : -1;
#pragma unroll
      for (int j = 0; j < HPT; ++j) {
        const int h = h0 + j;
        if (h < a.Hq)
          w[j].store(static_cast<T *>(a.q_out) + row * a.out_stride + static_cast<int64_t>(h) * a.D + d);
        else if (h < a.Hq + a.Hk && slot >= 0)
          w[j].store(static_cast<T *>(a.k_cache) + slot + (h - a.Hq) * a.head_stride + d);
      }
      continue;
    }
    u -= groups * keeps;
    // Eight elements of HPT heads of v.
    const int h0 = u / copies * HPT, d = u % copies * 8;
    Vec8<E> w[HPT];
#pragma unroll
    for (int j = 0; j < HPT; ++j)
      if (h0 + j < a.Hk)
        w[j].load(static_cast<const T *>(a.v) + row * a.v_stride + static_cast<int64_t>(h0 + j) * a.D + d);
    const int64_t slot = slot_offset(a, t);
    if (slot < 0) continue;
#pragma unroll
    for (int j = 0; j < HPT; ++j)
      if (h0 + j < a.Hk) w[j].store(static_cast<T *>(a.v_cache) + slot + (h0 + j) * a.head_stride + d);
  }
}

template <typename E, int HPT, bool INTERLEAVED>
cudaError_t launch_t(const RopeArgs &a, cudaStream_t stream) {
  const int groups = (a.Hq + a.Hk + HPT - 1) / HPT;
  const int units = groups * (a.r / 16 + (a.D - a.r) / 8) + (a.Hk + HPT - 1) / HPT * (a.D / 8);
  int per_block = 256 / units;
  if (per_block < 1) per_block = 1;
  const int64_t blocks = (static_cast<int64_t>(a.T) + per_block - 1) / per_block;
  rope_append_kernel<E, HPT, INTERLEAVED><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a, per_block, units);
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch_e(const RopeArgs &a, bool interleaved, cudaStream_t stream) {
  return interleaved ? launch_t<E, 2, true>(a, stream) : launch_t<E, 2, false>(a, stream);
}

}  // namespace

cudaError_t launch_rope_append(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                               const void *v, int64_t v_stride, int tokens, int q_heads,
                               const int *positions, int axes, const int *sections,
                               const float *cos_sin, int max_positions, int rotary_dim,
                               bool interleaved, const int *slots, void *q_out, int64_t out_stride,
                               const PagedPool &pool, cudaStream_t stream) {
  RopeArgs a{q, k, v, q_stride, k_stride, v_stride, out_stride, positions, slots, cos_sin, q_out,
             pool.k, pool.v, pool.page_stride, pool.head_stride, pool.token_stride,
             device_error_word(), pool.num_pages * pool.page_size, tokens, q_heads, pool.heads,
             pool.head_dim, rotary_dim, pool.page_size, max_positions, axes, {}};
  if (!a.err) return cudaErrorInvalidSymbol;
  int end = 0;
  for (int i = 0; i < axes; ++i) a.end[i] = end += sections[i];
  if (pool.type == kTypeBF16) return launch_e<ElemBF16>(a, interleaved, stream);
  if (pool.type == kTypeF16) return launch_e<ElemF16>(a, interleaved, stream);
  return launch_e<paged::ElemF32>(a, interleaved, stream);
}

}  // namespace qmm
