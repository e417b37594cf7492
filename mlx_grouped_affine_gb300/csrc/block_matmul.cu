// qmm_block_matmul: product of e4m3 codes, a scale per row and 128 columns on one side and
// per 128 x 128 block on the other.  One output a thread.
#include "common.cuh"

#include <cuda_fp8.h>

namespace qmm {
namespace {

__device__ __forceinline__ float2 widen2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return __half22float2(__half2(h));
}

__global__ void __launch_bounds__(256)
plain_kernel(const uint8_t *__restrict__ a, const float *__restrict__ as, int M,
             const uint8_t *__restrict__ w, const float *__restrict__ ws, int N, int K, int kb,
             void *__restrict__ y, int y_type) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x % 16;
  const int64_t m = static_cast<int64_t>(blockIdx.y) * 16 + threadIdx.x / 16;
  if (m >= M || n >= N) return;
  float sum = 0.0f;
  for (int b = 0; b < kb; ++b) {
    float part = 0.0f;
    for (int k = b * 128; k < min(K, b * 128 + 128); k += 4) {
      const uint32_t u = *reinterpret_cast<const uint32_t *>(a + m * K + k);
      const uint32_t v = *reinterpret_cast<const uint32_t *>(w + n * K + k);
      const float2 u0 = widen2(u & 0xFFFF), u1 = widen2(u >> 16), v0 = widen2(v & 0xFFFF), v1 = widen2(v >> 16);
      part = fmaf(u0.x, v0.x, part);
      part = fmaf(u0.y, v0.y, part);
      part = fmaf(u1.x, v1.x, part);
      part = fmaf(u1.y, v1.y, part);
    }
    sum = fmaf(as[m * kb + b] * ws[n / 128 * kb + b], part, sum);
  }
  const int64_t at = m * N + n;
  if (y_type == kTypeF32) static_cast<float *>(y)[at] = sum;
  else static_cast<uint16_t *>(y)[at] = y_type == kTypeBF16 ? ElemBF16::from_f32(sum) : ElemF16::from_f32(sum);
}

}  // namespace

cudaError_t launch_block_matmul(const uint8_t *a, const float *a_scales, int M, const uint8_t *w,
                                const float *w_scales, int N, int K, void *y, int y_type,
                                cudaStream_t stream) {
  const dim3 grid((N + 15) / 16, (M + 15) / 16);
  plain_kernel<<<grid, 256, 0, stream>>>(a, a_scales, M, w, w_scales, N, K, (K + 127) / 128, y, y_type);
  return cudaGetLastError();
}

}  // namespace qmm
