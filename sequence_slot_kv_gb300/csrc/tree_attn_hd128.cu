// tree_attn_hd128.cu -- the attention of drafted trees for head_dim 128.
#include "tree_attn.cuh"

namespace slotkv {

int launch_tree_hd128(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, uint32_t sms,
                     cudaStream_t stream) {
    return launch_tree_hd<128>(p, tmK, tmV, sms, stream);
}

}  // namespace slotkv
