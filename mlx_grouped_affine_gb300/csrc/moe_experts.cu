// qmm_moe_experts and qmm_moe_layer: gated feed-forward of each token's experts, in two
// kernels (moe_kernels.cuh): gate and up with silu, then down with the sum over a token's
// experts.  x that is not bf16 is first cut into bf16 planes that hold it exactly.
#include "moe_kernels.cuh"
#include "workspace.h"

namespace qmm {
namespace {

__global__ void __launch_bounds__(256)
planes_kernel(const void *__restrict__ x, int type, int64_t n, uint16_t *__restrict__ planes, int64_t plane, int count) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    store_planes(planes + i, plane, count, load_logit(x, type, i));
}

int64_t round128(int64_t n) { return (n + 127) / 128 * 128; }

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t hidden, int64_t inner) {
  return static_cast<size_t>(kWorkspaceAlign + 2 * 3 * round128(tokens * hidden) + 2 * 3 * round128(tokens * top_k * inner));
}

cudaError_t launch_moe_experts(const void *x, int x_type, int tokens, const Routing &r, const ExpertWeights &w,
                               void *y, int y_type, void *workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  MoeArgs a;
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidSymbol;
  const Workspace ws = aligned_workspace(workspace, workspace_bytes);
  const int64_t n = static_cast<int64_t>(tokens) * w.hidden;
  uint16_t *planes = reinterpret_cast<uint16_t *>(ws.base);
  a.route = r;
  a.w = w;
  a.tokens = tokens;
  a.y = y;
  a.y_type = y_type;
  a.wait_limit = wait_limit();
  a.x_plane = round128(n);
  a.x_planes = x_type == kTypeBF16 ? 1 : x_type == kTypeF16 ? 2 : 3;
  a.h = planes + 3 * a.x_plane;
  a.h_plane = round128(static_cast<int64_t>(tokens) * r.top_k * w.inner);
  a.h_planes = x_type == kTypeF32 ? 3 : 2;
  if (x_type == kTypeBF16) {
    a.x = static_cast<const uint16_t *>(x);
  } else {
    a.x = planes;
    const int64_t blocks = (n + 255) / 256, most = 8 * sm_count();
    planes_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, stream>>>(x, x_type, n, planes, a.x_plane,
                                                                                         a.x_planes);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  switch (w.bits) {
    case 1:
    case 2: return launch_moe_bits_1_2(a, stream);
    case 3: return launch_moe_bits_3(a, stream);
    case 4: return launch_moe_bits_4(a, stream);
    case 5:
    case 6: return launch_moe_bits_5_6(a, stream);
    case 8: return launch_moe_bits_8(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qmm
