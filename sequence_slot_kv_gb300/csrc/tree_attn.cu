// tree_attn.cu -- the attention of drafted trees (tree_attn.cuh) by head dim.
#include "tree_attn.cuh"

namespace slotkv {

int launch_tree_attn(int hd, const TreeParams& p, cudaStream_t stream) {
    return hd == 64    ? launch_tree_hd<64>(p, stream)
           : hd == 128 ? launch_tree_hd<128>(p, stream)
                       : launch_tree_hd<256>(p, stream);
}

}  // namespace slotkv
