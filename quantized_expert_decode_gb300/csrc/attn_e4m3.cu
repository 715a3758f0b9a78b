// attn_e4m3.cu — the streaming kernel of coli_attn_decode for E4M3 caches.
#include "attn_kernel.cuh"

namespace colimoe {

cudaError_t launch_attn_e4m3(const AttnParams &P, const AttnWork &W, int grid, cudaStream_t s) {
    return launch_dims<COLI_KV_E4M3>(P, W, grid, s);
}

}  // namespace colimoe
