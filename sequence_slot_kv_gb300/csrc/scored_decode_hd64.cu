// scored_decode_hd64.cu -- instantiations of the scored decode kernels (capped
// scores, distance bias, masks, shared prefixes) for head_dim 64 (G = 1..8
// query heads per kv head).  One translation unit per head dim so the builds
// run in parallel.
#include "decode_attn.cuh"
#include "decode_small.cuh"

namespace slotkv {

int launch_scored_hd64(int G, const ScoredDecodeParams& p, const CUtensorMap& tmK,
                       const CUtensorMap& tmV, unsigned ctas, bool small, cudaStream_t stream) {
    return small ? launch_small_hd<64, true>(G, p, stream)
                 : launch_hd<64, true>(G, p, tmK, tmV, ctas, stream);
}

}  // namespace slotkv
