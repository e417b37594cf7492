// qmm_block_quantize: e4m3 codes with one fp32 scale for each block of 128 columns, of
// one row or of 128 rows.
//
// scale = max(RN(amax / 448), 2^-126), code = the e4m3 value nearest to x / scale.  The
// quotient is taken as x * RN(1 / scale): two roundings of 2^-24, so it is within 2^-22 of
// the exact one and rounds to the same code unless a border between two codes is that near.
// Those elements (some 2^-17 of them) are compared with the border itself: border * scale
// has 5 + 24 bits and is exact in 64.  A division an element would cost more than the rest.
//
// Bound by memory: an element is read once and its code written once.  A thread holds 16
// consecutive elements (columns are a multiple of 16, so none is cut): 8 threads a row of a
// block, whose largest magnitude is joined by shuffles (and through shared memory over the
// 128 rows of a square block, whose elements wait in registers meanwhile).
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

// Whether q, within 2^-22 of a quotient, may lie on the other side of a border between two
// codes.  Codes of 2^-6 and more have 3 fraction bits, so a border has fraction bit 4 set and
// those below clear; smaller codes are multiples of 2^-9, their borders odd ones of 2^-10.
__device__ __forceinline__ bool near_border(float q) {
  const uint32_t b = __float_as_uint(q) & 0x7FFFFFFFu;
  if (b >= 0x3C800000u) return (b & 0xFFFFFu) - 0x7FFF8u <= 16u;
  const float u = fabsf(q) * 1024.0f, n = rintf(u);
  return fabsf(u - n) <= 1.9073486328125e-6f * 16.0f && (static_cast<int>(n) & 1);
}

// q moved to the side of its nearest border where x / s is.
__device__ __noinline__ float settle(float q, float x, float s) {
  const uint32_t b = __float_as_uint(q) & 0x7FFFFFFFu;
  const float t = b >= 0x3C800000u ? __uint_as_float((b & 0xFFF00000u) | 0x80000u)
                                   : rintf(fabsf(q) * 1024.0f) * 9.765625e-4f;
  const double d = fabs(static_cast<double>(x)) - static_cast<double>(t) * static_cast<double>(s);
  const uint32_t bits = __float_as_uint(t) + (d > 0.0 ? 1u : d < 0.0 ? 0xFFFFFFFFu : 0u);
  return copysignf(__uint_as_float(bits), x);
}

template <int T>
__device__ __forceinline__ uint4 codes_of(const Raw<T> &r, float s) {
  const float inv = __frcp_rn(s);
  uint32_t out[4];
  float q[16];
  bool slow = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    q[i] = r.at(i) * inv;
    slow |= near_border(q[i]);
  }
  if (slow) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (near_border(q[i])) q[i] = settle(q[i], r.at(i), s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    out[i] = lo | hi << 16;
  }
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
    const int64_t row = item / col_blocks;
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
  if (in) *reinterpret_cast<uint4 *>(codes + at) = codes_of(r, s);
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
    if (row < rows && col < cols) *reinterpret_cast<uint4 *>(codes + row * cols + col) = codes_of(r[i], s);
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
