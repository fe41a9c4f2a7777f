// prefill_paged.cu -- the attention of prefill.cuh over a paged cache: its blocks, or its tokens laid out before.
#include "prefill.cuh"

namespace da {

cudaError_t launch_prefill_paged(const PrefillParams& p, int grid, bool gathered, bool pdl, cudaStream_t stream) {
  return gathered ? launch_prefill_as<kGathered, true>(p, grid, pdl, stream) : launch_prefill_as<kPages16, true>(p, grid, pdl, stream);
}

}  // namespace da
