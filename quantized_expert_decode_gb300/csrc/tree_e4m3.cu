// tree_e4m3.cu — the streaming kernel of coli_attn_tree on e4m3 caches.
#include "tree_kernel.cuh"

namespace colimoe {

cudaError_t launch_tree_e4m3(const TreeParams &P, const TreeWork &W, const TreeMaps &maps, int grid, cudaStream_t s) {
    return launch_tree<COLI_KV_E4M3>(P, W, maps, grid, s);
}

}  // namespace colimoe
