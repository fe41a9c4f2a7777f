// prefill_paged.cu -- the attention of prefill.cuh over a paged cache, bf16 or e4m3.
#include "prefill.cuh"

namespace da {

cudaError_t launch_prefill_paged(const PrefillParams& p, int grid, bool kv8, bool pdl, cudaStream_t stream) {
  return kv8 ? launch_prefill_as<kPages8, true>(p, grid, pdl, stream) : launch_prefill_as<kPages16, true>(p, grid, pdl, stream);
}

}  // namespace da
