// attn_f16.cu — the streaming kernel of coli_attn_decode for F16 caches.
#include "attn_kernel.cuh"

namespace colimoe {

cudaError_t launch_attn_f16(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s) {
    return launch_dims<COLI_KV_F16>(P, W, grid, s);
}

}  // namespace colimoe
