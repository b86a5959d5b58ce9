// Instantiations of the sm_103a cross-attention forward kernel for head dimension 96.
#include "fa2_kernel.cuh"

namespace fa2 {
template cudaError_t launch_cross_fwd<96, false>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                              const CUtensorMap&, const CrossParams&, int, cudaStream_t);
template cudaError_t launch_cross_fwd<96, true>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                             const CUtensorMap&, const CrossParams&, int, cudaStream_t);
}  // namespace fa2
