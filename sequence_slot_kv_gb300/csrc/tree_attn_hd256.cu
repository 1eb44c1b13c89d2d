// tree_attn_hd256.cu -- the attention of drafted trees for head_dim 256.
#include "tree_attn.cuh"

namespace slotkv {

int launch_tree_hd256(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, uint32_t sms,
                     cudaStream_t stream) {
    return launch_tree_hd<256>(p, tmK, tmV, sms, stream);
}

}  // namespace slotkv
