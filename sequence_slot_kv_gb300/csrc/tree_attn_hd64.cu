// tree_attn_hd64.cu -- the attention of drafted trees for head_dim 64.
#include "tree_attn.cuh"

namespace slotkv {

int launch_tree_hd64(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, uint32_t sms,
                     cudaStream_t stream) {
    return launch_tree_hd<64>(p, tmK, tmV, sms, stream);
}

}  // namespace slotkv
