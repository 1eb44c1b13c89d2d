// scored_prefill_hd64.cu -- instantiations of the scored tensor-core prefill
// (capped scores, distance bias, masks, the prefix pass of a shared call) for
// head_dim 64 (G = 1..8 query heads per kv head).  One translation unit per
// head dim so the builds run in parallel.
#include "prefill_tc.cuh"

namespace slotkv {

int launch_scored_prefill_hd64(int G, const ScoredPrefillParams& p, const CUtensorMap& tmK,
                               const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream) {
    return launch_prefill_hd<64, true>(G, p, tmK, tmV, ctas, stream);
}

}  // namespace slotkv
