// qmm_moe_experts and qmm_moe_layer: gated feed-forward of each token's experts.  One warp
// an output: silu(gate) * up of one slot and inner row, then one token and hidden row.
#include "moe_route.cuh"
#include "workspace.h"

namespace qmm {
namespace {

__device__ __forceinline__ float load_as_f32(const void *p, int type, int64_t at) {
  return load_logit(p, type, at);
}

__device__ __forceinline__ float weight_at(const ExpertWeights &w, int part, int64_t row, int cols, int k) {
  const int64_t bit = static_cast<int64_t>(k) * w.bits;
  const uint32_t *p = w.w[part] + row * (static_cast<int64_t>(cols) * w.bits / 32) + bit / 32;
  const int sh = bit % 32;
  uint32_t c = p[0] >> sh;
  if (sh + w.bits > 32) c |= p[1] << (32 - sh);
  c &= (1u << w.bits) - 1u;
  const int64_t g = row * (cols / w.group) + k / w.group;
  return fmaf(load_as_f32(w.scales[part], w.sb_type, g), static_cast<float>(c),
              load_as_f32(w.biases[part], w.sb_type, g));
}

__global__ void __launch_bounds__(256)
plain_route(const __grid_constant__ Routing r, int tokens, int experts, int *ids, float *weights, unsigned *err) {
  const int lane = threadIdx.x % 32;
  for (int t = threadIdx.x / 32; t < tokens; t += 8) {
    int id = 0;
    float weight = 0;
    if (r.logits) route_row<32>(r, experts, t, lane, id, weight);
    else if (lane < r.top_k) id = r.ids[t * r.top_k + lane], weight = r.weights[t * r.top_k + lane];
    if (lane < r.top_k) {
      if (id < 0 || id >= experts) {
        atomicOr(err, kErrIndexBit);
        id = 0, weight = 0.0f;
      }
      ids[t * r.top_k + lane] = id;
      weights[t * r.top_k + lane] = weight;
    }
  }
}

__global__ void __launch_bounds__(256)
plain_gate_up(const void *__restrict__ x, int x_type, const __grid_constant__ ExpertWeights w, int top_k,
              const int *ids, const float *weights, float *__restrict__ h) {
  const int slot = blockIdx.y, row = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (row >= w.inner || weights[slot] == 0.0f) return;
  const int64_t e = ids[slot], t = slot / top_k;
  float g = 0, u = 0;
  for (int k = lane; k < w.hidden; k += 32) {
    const float v = load_as_f32(x, x_type, t * w.hidden + k);
    g = fmaf(weight_at(w, 0, e * w.inner + row, w.hidden, k), v, g);
    u = fmaf(weight_at(w, 1, e * w.inner + row, w.hidden, k), v, u);
  }
  g = warp_sum(g), u = warp_sum(u);
  if (lane == 0) h[static_cast<int64_t>(slot) * w.inner + row] = g / (1.0f + expf(-g)) * u;
}

__global__ void __launch_bounds__(256)
plain_down(const float *__restrict__ h, const __grid_constant__ ExpertWeights w, int top_k, const int *ids,
           const float *weights, void *__restrict__ y, int y_type) {
  const int t = blockIdx.y, row = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (row >= w.hidden) return;
  float sum = 0;
  for (int j = 0; j < top_k; ++j) {
    const int slot = t * top_k + j;
    if (weights[slot] == 0.0f) continue;
    const int64_t e = ids[slot];
    float z = 0;
    for (int k = lane; k < w.inner; k += 32)
      z = fmaf(weight_at(w, 2, e * w.hidden + row, w.inner, k), h[static_cast<int64_t>(slot) * w.inner + k], z);
    sum = fmaf(weights[slot], warp_sum(z), sum);
  }
  if (lane != 0) return;
  const int64_t at = static_cast<int64_t>(t) * w.hidden + row;
  if (y_type == kTypeF32) static_cast<float *>(y)[at] = sum;
  else static_cast<uint16_t *>(y)[at] = y_type == kTypeBF16 ? ElemBF16::from_f32(sum) : ElemF16::from_f32(sum);
}

}  // namespace

size_t moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t hidden, int64_t inner) {
  return static_cast<size_t>(kWorkspaceAlign + 8 * kMoeMaxSlots + 6 * tokens * hidden + 128 + 6 * tokens * top_k * inner);
}

cudaError_t launch_moe_experts(const void *x, int x_type, int tokens, const Routing &r, const ExpertWeights &w,
                               void *y, int y_type, void *workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  unsigned *err = device_error_word();
  if (!err) return cudaErrorInvalidSymbol;
  const Workspace ws = aligned_workspace(workspace, workspace_bytes);
  int *ids = reinterpret_cast<int *>(ws.base);
  float *weights = reinterpret_cast<float *>(ws.base + 4 * kMoeMaxSlots);
  float *h = reinterpret_cast<float *>(ws.base + 8 * kMoeMaxSlots);
  plain_route<<<1, 256, 0, stream>>>(r, tokens, w.experts, ids, weights, err);
  plain_gate_up<<<dim3((w.inner + 7) / 8, tokens * r.top_k), 256, 0, stream>>>(x, x_type, w, r.top_k, ids, weights, h);
  plain_down<<<dim3((w.hidden + 7) / 8, tokens), 256, 0, stream>>>(h, w, r.top_k, ids, weights, y, y_type);
  return cudaGetLastError();
}

}  // namespace qmm
