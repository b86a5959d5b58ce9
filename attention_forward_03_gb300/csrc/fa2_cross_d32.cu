// Instantiations of the sm_103a cross-attention forward kernel for head dimension 32.
#include "fa2_kernel.cuh"

namespace fa2 {
template cudaError_t launch_cross_fwd<32, false>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                              const CUtensorMap&, const CrossParams&, int, cudaStream_t);
template cudaError_t launch_cross_fwd<32, true>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                             const CUtensorMap&, const CrossParams&, int, cudaStream_t);
}  // namespace fa2
