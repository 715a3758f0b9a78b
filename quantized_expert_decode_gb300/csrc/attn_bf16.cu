// attn_bf16.cu — the streaming kernel of coli_attn_decode for BF16 caches.
#include "attn_kernel.cuh"

namespace colimoe {

cudaError_t launch_attn_bf16(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s) {
    return launch_dims<COLI_KV_BF16>(P, W, grid, s);
}

}  // namespace colimoe
