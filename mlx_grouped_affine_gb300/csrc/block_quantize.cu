// qmm_block_quantize: e4m3 codes with one fp32 scale for each block of 128 columns, of
// one row or of 128 rows.
//
// scale = max(RN(amax / 448), 2^-126), code = the e4m3 value nearest to x / scale.  The
// quotient is taken as x * RN(1 / scale): two roundings of 2^-24, so it is within 2^-22 of
// the exact one and rounds to the same code unless a border between two codes is that near.
// Those elements are compared with the border itself, border * scale with x in one fused
// multiply-add.  A division an element would cost more than the rest.  Of normal
// values they are one in 87000 in fp32, but one in 1600 in fp16 and one in 180 in bf16, whose
// quotients, ratios of two short numbers, often lie on a border exactly.
//
// Bound by memory: an element is read once and its code written once.  A thread holds 16
// consecutive elements (columns are a multiple of 16, so none is cut): 8 threads a row of a
// block, whose largest magnitude is joined by shuffles (and through shared memory over the
// 128 rows of a square block, whose elements wait in registers meanwhile).  [11008, 4096] fp32
// in square blocks 42.0 us, 5.4 TB/s, 0.79 of the copy rate; 16 x 4096 bf16 by rows 3.3 us, the
// launch and one chain of load, shuffles and codes.  16-bit elements are bound by instructions:
// the same in fp16 42.4 us, in bf16 55.7 (settled_codes); 2048 x 4096 by rows 13.3 us in bf16, 8.7
// in fp32.
#include "common.cuh"

#include <cuda_fp8.h>

namespace qmm {
namespace {

constexpr float kMax = 448.0f;           // largest e4m3 value
constexpr float kMinScale = 1.1754943508222875e-38f;  // 2^-126
constexpr int kThreads = 256;
constexpr int kRun = 16;  // elements of a thread
constexpr int kLanes = 128 / kRun;

template <int T>
struct Raw {  // 16 elements as loaded
  uint4 v[T == kTypeF32 ? 4 : 2];
  __device__ __forceinline__ void load(const void *x, int64_t at) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(x) + at * (T == kTypeF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (T == kTypeF32 ? 4 : 2); ++i) v[i] = __ldcs(p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (T == kTypeF32 ? 4 : 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
    if constexpr (T == kTypeF32) return __uint_as_float(w[i]);
    const uint32_t h = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu;
    if constexpr (T == kTypeBF16) return bf16_bits_to_f32(h);
    return ElemF16::to_f32(h);
  }
  // The largest magnitude's bits; a NaN's are above all others.
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(v);
    uint32_t m = 0;
    if constexpr (T == kTypeF32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    } else {
      // two 16-bit patterns at a time
#pragma unroll
      for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      m = max(m >> 16, m & 0xFFFFu);
      m = __float_as_uint(T == kTypeBF16 ? bf16_bits_to_f32(m) : ElemF16::to_f32(m));
    }
    return m;
  }
};

__device__ __forceinline__ float scale_of(uint32_t top) {
  const float s = __fdiv_rn(__uint_as_float(top), kMax);
  return s < kMinScale ? kMinScale : s;  // (a NaN stays)
}

// |q| as a number whose codes are 2^-3 of its power of two apart: codes below 2^-6 are
// multiples of 2^-9, as those in [2^-6, 2^-5) are.  A border between two codes then has
// fraction bit 4 set and those below clear, whatever its size.
__device__ __forceinline__ float on_grid(float q) { return fabsf(q) < 0.015625f ? fabsf(q) + 0.015625f : fabsf(q); }

// At most kNear where on_grid(q) is within 4 units of its last place of a border (it is off
// by 2.5 at most: two roundings of half a unit of a number up to twice as large, and a third).
constexpr uint32_t kNear = 8;
__device__ __forceinline__ uint32_t off_border(float q) { return (__float_as_uint(on_grid(q)) - 0x7FFFCu) & 0xFFFFFu; }

// q moved to the side of its border where x / s is.
__device__ __forceinline__ float settle(float q, float x, float s) {
  const float up = on_grid(q), border = __uint_as_float((__float_as_uint(up) & 0xFFF00000u) | 0x80000u);
  const float t = fabsf(q) < 0.015625f ? border - 0.015625f : border;
  // t s has 5 + 24 bits: the fused multiply-add gives the difference's sign, after a factor
  // that keeps small ones from vanishing.
  const float by = s < 1.0f ? 1099511627776.0f : 1.0f;  // 2^40
  const float d = fmaf(-t, s * by, fabsf(x) * by);
  const uint32_t bits = __float_as_uint(t) + (d > 0.0f ? 1u : d < 0.0f ? 0xFFFFFFFFu : 0u);
  return copysignf(__uint_as_float(bits), x);
}

__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The 16 codes again, element by element, for a thread that met a border (one in 5500 in fp32,
// 106 in fp16, 14 in bf16).
// Rolled up: nothing here should cost the others instruction cache.
__device__ __noinline__ uint4 settled_codes(const void *x, int type, int64_t at, float s, float inv) {
  uint32_t out[4] = {};
#pragma unroll 1
  for (int i = 15; i >= 0; --i) {
    const uint32_t h = type == kTypeF32 ? 0u : static_cast<const uint16_t *>(x)[at + i];
    const float v = type == kTypeF32    ? static_cast<const float *>(x)[at + i]
                    : type == kTypeBF16 ? bf16_bits_to_f32(h)
                                        : ElemF16::to_f32(h);
    float q = v * inv;
    if (off_border(q) <= kNear) q = settle(q, v, s);
    // shift the codes up by one byte and put this one below them
    out[3] = out[3] << 8 | out[2] >> 24;
    out[2] = out[2] << 8 | out[1] >> 24;
    out[1] = out[1] << 8 | out[0] >> 24;
    out[0] = out[0] << 8 | (code2(q, 0.0f) & 0xFFu);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int T>
__device__ __forceinline__ uint4 codes_of(const Raw<T> &r, float s, const void *x, int64_t at) {
  const float inv = __frcp_rn(s);
  uint32_t out[4], nearest = 0xFFFFFu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      q[k] = r.at(4 * i + k) * inv;
      nearest = min(nearest, off_border(q[k]));
    }
    out[i] = code2(q[0], q[1]) | code2(q[2], q[3]) << 16;
  }
  if (nearest <= kNear) return settled_codes(x, T, at, s, inv);
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// A scale per row and 128 columns: 8 threads a block, 32 blocks a thread block.
template <int T>
__global__ void __launch_bounds__(kThreads)
rows_kernel(const void *__restrict__ x, int64_t total, uint32_t col_blocks, uint32_t cols,
            uint8_t *__restrict__ codes, float *__restrict__ scales) {
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  Raw<T> r;
  int64_t at = 0;
  bool in = item < total;
  if (in) {
    // (a division of 64 bits would cost more than the codes)
    const int64_t row = total < (int64_t(1) << 31) ? static_cast<uint32_t>(item) / col_blocks : item / col_blocks;
    const uint32_t col = static_cast<uint32_t>(item - row * col_blocks) * 128u + lane * kRun;
    at = row * cols + col;
    in = col < cols;
  }
  if (in) r.load(x, at);
  else r.zero();
  uint32_t top = r.top();
#pragma unroll
  for (int d = 1; d < kLanes; d *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  const float s = scale_of(top);
  if (in) *reinterpret_cast<uint4 *>(codes + at) = codes_of(r, s, x, at);
  if (item < total && lane == 0) scales[item] = s;
}

// A scale per 128 x 128 block: one thread block each, 32 rows at a time.
template <int T>
__global__ void __launch_bounds__(kThreads)
square_kernel(const void *__restrict__ x, int64_t rows, uint32_t cols, uint32_t col_blocks,
              uint8_t *__restrict__ codes, float *__restrict__ scales) {
  __shared__ uint32_t tops[kThreads / 32];
  constexpr int kStep = kThreads / kLanes, kParts = 128 / kStep;
  const uint32_t by = blockIdx.x / col_blocks, bx = blockIdx.x - by * col_blocks;
  const int64_t row0 = static_cast<int64_t>(by) * 128 + threadIdx.x / kLanes;
  const uint32_t col = bx * 128u + threadIdx.x % kLanes * kRun;
  Raw<T> r[kParts];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const int64_t row = row0 + i * kStep;
    if (row < rows && col < cols) r[i].load(x, row * cols + col);
    else r[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kParts; ++i) top = max(top, r[i].top());
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) top = max(top, tops[i]);
  const float s = scale_of(top);
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const int64_t row = row0 + i * kStep;
    if (row < rows && col < cols) *reinterpret_cast<uint4 *>(codes + row * cols + col) = codes_of(r[i], s, x, row * cols + col);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

template <int T>
cudaError_t launch(const void *x, int64_t rows, int64_t cols, bool square, uint8_t *codes, float *scales,
                   cudaStream_t stream) {
  const int64_t col_blocks = (cols + 127) / 128;
  const int64_t blocks = square ? (rows + 127) / 128 * col_blocks
                                : (rows * col_blocks + kThreads / kLanes - 1) / (kThreads / kLanes);
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (square)
    square_kernel<T><<<grid, kThreads, 0, stream>>>(x, rows, static_cast<uint32_t>(cols),
                                                    static_cast<uint32_t>(col_blocks), codes, scales);
  else
    rows_kernel<T><<<grid, kThreads, 0, stream>>>(x, rows * col_blocks, static_cast<uint32_t>(col_blocks),
                                                  static_cast<uint32_t>(cols), codes, scales);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_quantize(const void *x, int x_type, int64_t rows, int64_t cols, bool square,
                                  uint8_t *codes, float *scales, cudaStream_t stream) {
  switch (x_type) {
    case kTypeF32: return launch<kTypeF32>(x, rows, cols, square, codes, scales, stream);
    case kTypeBF16: return launch<kTypeBF16>(x, rows, cols, square, codes, scales, stream);
    default: return launch<kTypeF16>(x, rows, cols, square, codes, scales, stream);
  }
}

}  // namespace qmm
