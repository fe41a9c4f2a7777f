// prefill.cu -- the attention of prefill.cuh over packed prompts, whole or with a window.
#include "prefill.cuh"

namespace da {

cudaError_t launch_prefill(const PrefillParams& p, int grid, bool pdl, cudaStream_t stream) {
  return launch_prefill_as<kPackedKeys, false>(p, grid, pdl, stream);
}
cudaError_t launch_prefill_window(const PrefillParams& p, int grid, bool pdl, cudaStream_t stream) {
  return launch_prefill_as<kPackedKeys, true>(p, grid, pdl, stream);
}

}  // namespace da
