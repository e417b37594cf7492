// qmm_moe_route: top experts and weights, one warp a token.  A lane keeps every 32nd logit
// as an ordered integer in a register; each choice is the warp's largest of them and, of
// equal ones, the lowest expert: two warp reductions, one for 16-bit logits, which share a word
// with their expert.  8192 tokens over 256 experts, top 8, bf16, in 6.9 us (two more with two
// reductions; fp32 8.4), bound by integer instructions: every choice looks at all of a lane's
// entries again (fp32 over 1024 experts 23.8 us).  16 over 128 in 2.8 us, the launch and eight
// choices.
#include "moe_route.cuh"

namespace qmm {
namespace {

constexpr int kWarps = 8;

template <int NV, bool PACKED>
__global__ void __launch_bounds__(32 * kWarps)
route_kernel(const __grid_constant__ Routing r, int64_t tokens, int experts, int *__restrict__ ids,
             float *__restrict__ weights) {
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (row >= tokens) return;
  int id;
  float weight;
  route_row<NV, PACKED>(r, experts, row, lane, id, weight);
  if (lane < r.top_k) {
    ids[row * r.top_k + lane] = id;
    weights[row * r.top_k + lane] = weight;
  }
}

template <int NV>
cudaError_t launch(const Routing &r, int64_t tokens, int experts, int *ids, float *weights,
                   cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((tokens + kWarps - 1) / kWarps);
  if (r.type == kTypeF32) route_kernel<NV, false><<<grid, 32 * kWarps, 0, stream>>>(r, tokens, experts, ids, weights);
  else route_kernel<NV, true><<<grid, 32 * kWarps, 0, stream>>>(r, tokens, experts, ids, weights);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_route(const Routing &r, int64_t tokens, int experts, int *ids, float *weights,
                             cudaStream_t stream) {
  if (experts <= 32) return launch<1>(r, tokens, experts, ids, weights, stream);
  if (experts <= 64) return launch<2>(r, tokens, experts, ids, weights, stream);
  if (experts <= 128) return launch<4>(r, tokens, experts, ids, weights, stream);
  if (experts <= 256) return launch<8>(r, tokens, experts, ids, weights, stream);
  if (experts <= 512) return launch<16>(r, tokens, experts, ids, weights, stream);
  return launch<32>(r, tokens, experts, ids, weights, stream);
}

}  // namespace qmm
