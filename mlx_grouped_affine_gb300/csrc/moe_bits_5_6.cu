// The expert kernels for codes of 5 and 6 bits.
#include "moe_kernels.cuh"

namespace qmm {

cudaError_t launch_moe_bits_5_6(const MoeArgs &a, cudaStream_t stream) {
  return a.w.bits == 5 ? launch_moe_bits<5>(a, stream) : launch_moe_bits<6>(a, stream);
}

}  // namespace qmm
