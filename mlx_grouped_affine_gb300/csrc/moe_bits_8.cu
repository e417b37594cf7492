// The expert kernels for codes of 8 bits.
#include "moe_kernels.cuh"

namespace qmm {

cudaError_t launch_moe_bits_8(const MoeArgs &a, cudaStream_t stream) {
  return launch_moe_bits<8>(a, stream);
}

}  // namespace qmm
