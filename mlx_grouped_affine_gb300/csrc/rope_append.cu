// Rotary positions on q and k, and K and V into the paged cache, in one pass.
//
// Pair i of a head (x1, x2) turns by the angle of position pos[axis(i)] and
// frequency i: (x1 c - x2 s, x2 c + x1 s), c and s from the caller's fp32
// table, products and sums in fp32, one rounding to the element type.  The
// pairs are (i, i + r/2) or (2i, 2i + 1); axis(i) follows from the sections.
//
// Nothing is read twice but the table's row, so bytes bound it: q, k, v read
// once, q, K, V written once, 16 bytes a lane.  A thread has one place in a token
// (eight pairs of a head, or eight elements that pass through) and walks a few
// tokens with it: where its elements come from and go to is worked out once, a
// token costs it a few adds.  8192 tokens of 40 heads of 128 with three axes:
// 206 MB in 40 us, 5.1 TB/s, 0.75 of the measured copy rate; 16 tokens: 2.1 us,
// the launch.
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
struct Vec8 {  // eight elements in their own type
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

// The cosines and sines of pairs i0 .. i0 + 7 for token t; a bit for each pair
// whose position is outside the table.  `axis` is the first pair's.  Where the
// axis changes among the eight, the next axis's row is read whole too and its
// pairs replace the first's.
__device__ __forceinline__ unsigned angles(const RopeArgs &a, int t, int i0, int axis, float (&c)[8],
                                           float (&s)[8]) {
  const int half = a.r / 2;
  auto row = [&](int x, float (&cx)[8], float (&sx)[8]) {
    const int pos = __ldg(a.positions + static_cast<int64_t>(x) * a.T + t);
    const bool ok = static_cast<unsigned>(pos) < static_cast<unsigned>(a.max_pos);
    const float *p = a.table + static_cast<int64_t>(ok ? pos : 0) * a.r + i0;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const float4 cv = __ldg(reinterpret_cast<const float4 *>(p + e));
      const float4 sv = __ldg(reinterpret_cast<const float4 *>(p + half + e));
      cx[e] = cv.x; cx[e + 1] = cv.y; cx[e + 2] = cv.z; cx[e + 3] = cv.w;
      sx[e] = sv.x; sx[e + 1] = sv.y; sx[e + 2] = sv.z; sx[e + 3] = sv.w;
    }
    return ok ? 0u : 0xFFu;
  };
  unsigned outside = row(axis, c, s);
#pragma unroll 1
  for (int x = axis; x < a.axes - 1 && a.end[x] < i0 + 8; ++x) {
    const int from = a.end[x] - i0;  // the next axis's pairs
    float cx[8], sx[8];
    const unsigned bad = row(x + 1, cx, sx);
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      if (e >= from) {
        c[e] = cx[e];
        s[e] = sx[e];
      }
    }
    const unsigned mine = 0xFFu << from;
    outside = (outside & ~mine) | (bad & mine);
  }
  return outside;
}

// Measured on 8192 tokens of 40 heads of 128, three axes: 64 threads and at most
// 64 registers (16 blocks an SM) 40 us, 128 threads 42, 48 registers (spills) 54.
constexpr int kThreads = 64;

template <typename E, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 16) rope_append_kernel(const __grid_constant__ RopeArgs a, int units,
                                                               int tokens) {
  using T = typename Elem<E>::type;
  const int half = a.r / 2, turns = a.r / 16, keeps = (a.D - a.r) / 8, copies = a.D / 8, heads = a.Hq + a.Hk;
  int u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= units) return;
  // The thread's place: a turn (i0, its first pair), a copy of q or k past the
  // turned elements, or a copy of v.
  const bool turn = u < heads * turns;
  int h, d0, d1, i0 = 0;  // head, and the first elements of its two (one) vectors
  bool v = false;
  if (turn) {
    h = u / turns;
    i0 = (u - h * turns) * 8;
    d0 = INTERLEAVED ? 2 * i0 : i0;
    d1 = INTERLEAVED ? 2 * i0 + 8 : half + i0;
  } else if ((u -= heads * turns) < heads * keeps) {
    h = u / keeps;
    d0 = d1 = a.r + (u - h * keeps) * 8;
  } else {
    u -= heads * keeps;
    h = u / copies;
    d0 = d1 = (u - h * copies) * 8;
    v = true;
  }
  const bool query = !v && h < a.Hq;
  if (!v && !query) h -= a.Hq;
  const T *src = static_cast<const T *>(v ? a.v : query ? a.q : a.k) + static_cast<int64_t>(h) * a.D;
  const int64_t src_stride = v ? a.v_stride : query ? a.q_stride : a.k_stride;
  T *dst = query ? static_cast<T *>(a.q_out) + static_cast<int64_t>(h) * a.D
                 : static_cast<T *>(v ? a.v_cache : a.k_cache) + h * a.head_stride;
  int axis = 0;
  while (axis < a.axes - 1 && i0 >= a.end[axis]) ++axis;
  const int t0 = blockIdx.y * tokens, t1 = t0 + min(tokens, a.T - t0);
#pragma unroll 1
  for (int t = t0; t < t1; ++t) {
    const T *from = src + t * src_stride;
    Vec8<E> lo, hi;
    lo.load(from + d0);
    if (turn) hi.load(from + d1);
    int64_t to = t * a.out_stride;
    if (!query) to = slot_offset(a, t);
    if (turn) {
      float c[8], s[8], x0[8], x1[8];
      const unsigned outside = angles(a, t, i0, axis, c, s);
      if (outside) atomicOr(a.err, kErrIndexBit);
      lo.get(x0);
      hi.get(x1);
      // Pair e is (y0, y1) of the two vectors, or consecutive elements of them.
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float &y0 = INTERLEAVED ? (e < 4 ? x0[2 * e] : x1[2 * e - 8]) : x0[e];
        float &y1 = INTERLEAVED ? (e < 4 ? x0[2 * e + 1] : x1[2 * e - 7]) : x1[e];
        const float z0 = y0, z1 = y1;
        y0 = z0 * c[e] - z1 * s[e];
        y1 = z1 * c[e] + z0 * s[e];
        if (outside >> e & 1u) y0 = y1 = 0.f;  // whatever q and k hold
      }
      lo.set(x0);
      hi.set(x1);
    }
    if (to < 0) continue;
    lo.store(dst + to + d0);
    if (turn) hi.store(dst + to + d1);
  }
}

template <typename E, bool INTERLEAVED>
cudaError_t launch_t(const RopeArgs &a, cudaStream_t stream) {
  const int heads = a.Hq + a.Hk;
  const int units = heads * (a.r / 16 + (a.D - a.r) / 8) + a.Hk * (a.D / 8);
  const unsigned columns = (units + kThreads - 1) / kThreads;
  // Tokens of a thread: up to 8, as long as the SMs have eight blocks each.  Measured
  // on 16 / 1021 / 8192 tokens: this rule 2.1 / 3.4 / 40 us, always one 2.1 / 3.7 / 54,
  // always eight 6.0 / 6.7 / 40, up to 32 2.1 / 3.4 / 46.
  int tokens = static_cast<int>(static_cast<int64_t>(a.T) * columns / (8 * sm_count()));
  tokens = tokens < 1 ? 1 : tokens > 8 ? 8 : tokens;
  const int64_t T = a.T;
  while ((T + tokens - 1) / tokens > 65535) tokens *= 2;
  const dim3 grid(columns, static_cast<unsigned>((T + tokens - 1) / tokens));
  rope_append_kernel<E, INTERLEAVED><<<grid, kThreads, 0, stream>>>(a, units, tokens);
  return cudaGetLastError();
}

template <typename E>
cudaError_t launch_e(const RopeArgs &a, bool interleaved, cudaStream_t stream) {
  return interleaved ? launch_t<E, true>(a, stream) : launch_t<E, false>(a, stream);
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
