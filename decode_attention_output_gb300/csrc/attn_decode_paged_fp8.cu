// attn_decode_paged_fp8.cu -- instantiations of the attention kernel over a paged fp8 (e4m3)
// KV cache with a scale per token and KV head: head dim 128, 128-token tiles, 4-stage ring.
#include "attn_decode.cuh"

namespace da {

cudaError_t launch_attention_paged_fp8(const AttnParams& p, int grid, int nb, cudaStream_t stream) {
  return nb == 1 ? launch_one<1, false, 4, 0, kHeadDim, true, true>(p, grid, stream)
                 : launch_one<2, false, 4, 0, kHeadDim, true, true>(p, grid, stream);
}

}  // namespace da
