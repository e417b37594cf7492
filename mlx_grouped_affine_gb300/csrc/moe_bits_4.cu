// The expert kernels for codes of 4 bits.
#include "moe_kernels.cuh"

namespace qmm {

cudaError_t launch_moe_bits_4(const MoeArgs &a, cudaStream_t stream) {
  return launch_moe_bits<4>(a, stream);
}

}  // namespace qmm
