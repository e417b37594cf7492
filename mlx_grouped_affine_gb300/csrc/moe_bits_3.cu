// The expert kernels for codes of 3 bits.
#include "moe_kernels.cuh"

namespace qmm {

cudaError_t launch_moe_bits_3(const MoeArgs &a, cudaStream_t stream) {
  return launch_moe_bits<3>(a, stream);
}

}  // namespace qmm
