// Attention over a paged cache on the tensor cores (fa2_paged_kernel.cuh), head dimension 96.
#include "fa2_paged_kernel.cuh"

namespace fa2 {

template cudaError_t launch_paged_tiles<96, true>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                                  const PagedTileParams&, int, cudaStream_t);
template cudaError_t launch_paged_tiles<96, false>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                                   const PagedTileParams&, int, cudaStream_t);

}  // namespace fa2
