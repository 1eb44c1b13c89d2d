// scored_decode_hd256.cu -- instantiations of the scored decode kernels (capped
// scores, distance bias, masks, shared prefixes) for head_dim 256 (G = 1..8
// query heads per kv head).  One translation unit per head dim so the builds
// run in parallel.
#include "decode_attn.cuh"
#include "decode_small.cuh"

namespace slotkv {

int launch_scored_hd256(int G, const ScoredDecodeParams& p, const CUtensorMap& tmK,
                       const CUtensorMap& tmV, unsigned ctas, bool small, ScoredPart part,
                       cudaStream_t stream) {
    if (!small) return launch_hd<256, true>(G, p, tmK, tmV, ctas, stream, part);
    if (part == ScoredPart::plan) return 0;  // one kernel, no plan
    return launch_small_hd<256, true>(G, p, stream);
}

}  // namespace slotkv
