// The expert kernels for codes of 1 and 2 bits.
#include "moe_kernels.cuh"

namespace qmm {

cudaError_t launch_moe_bits_1_2(const MoeArgs &a, cudaStream_t stream) {
  return a.w.bits == 1 ? launch_moe_bits<1>(a, stream) : launch_moe_bits<2>(a, stream);
}

}  // namespace qmm
