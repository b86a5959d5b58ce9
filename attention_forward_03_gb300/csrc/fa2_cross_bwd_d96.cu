// Instantiations of the sm_103a cross-attention backward kernel for head dimension 96.
#include "fa2_bwd_kernel.cuh"

namespace fa2 {
template cudaError_t launch_cross_bwd<96, false>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                              const CUtensorMap&, const CUtensorMap&, const CrossBwdParams&, int,
                                              cudaStream_t);
template cudaError_t launch_cross_bwd<96, true>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                             const CUtensorMap&, const CUtensorMap&, const CrossBwdParams&, int,
                                             cudaStream_t);
}  // namespace fa2
