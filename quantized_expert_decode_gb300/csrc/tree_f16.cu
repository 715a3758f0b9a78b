// tree_f16.cu — the streaming kernel of coli_attn_tree on f16 caches.
#include "tree_kernel.cuh"

namespace colimoe {

cudaError_t launch_tree_f16(const TreeParams &P, const TreeWork &W, const TreeMaps &maps, int grid, cudaStream_t s) {
    return launch_tree<COLI_KV_F16>(P, W, maps, grid, s);
}

}  // namespace colimoe
