// tree_attn.h -- launch parameters of the attention of drafted trees
// (tree_attn.cuh).  Plain data only.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "params.h"

namespace slotkv {

// Nodes a request's tree may have, and the words of a set of them.
constexpr uint32_t kTreeNodes = 256, kTreeWords = kTreeNodes / 32;

struct TreeParams {
    const float* q;          // [n_tok][n_head][hd]
    const float* k_new;      // [n_tok][n_kv_head][hd]
    const float* v_new;
    const uint32_t* slots;   // [n_req], or null: paged
    const uint32_t* block_tables;  // [n_req][bt_stride]
    const uint32_t* past;    // [n_req]
    const uint32_t* starts;  // [n_req + 1]
    const uint32_t* parents; // [n_tok]
    const float* q_norm_w;   // [hd]
    const float* k_norm_w;
    const float* inv_freq;   // [hd/2]
    const float* sinks;      // [n_head] or null
    float* out;              // [n_tok][n_head][hd]
    float* K;                // [n_slots][slot_ctx][n_kv_head][hd]
    float* V;
    float* q_rot;            // workspace [n_tok][n_head][hd]: normed, rotated, scaled q
    uint32_t* req_of;        // workspace [n_tok]: the node's request, kTreeSkip: skipped
    uint32_t* depth;         // workspace [n_tok]
    uint32_t* below;         // workspace [n_tok][kTreeWords]: the nodes that attend it (words past the
                             // request's nodes are not written)
    float* part;             // workspace: partial results, two of a unit's rows per CTA [rows][hd]
    float* part_ml;          // and their (m, l)
    uint32_t* plan;          // workspace [CTAs][kTreePlan]: where each CTA's part of the work begins
    uint32_t* join;          // workspace [CTAs][kTreeJoin]: the unit that begins in a CTA and ends in another
    uint32_t* status;        // sticky SLOTKV_DEV_* flags
    uint32_t n_slots, slot_ctx, bt_stride, n_head, n_kv_head, n_req, n_tok;
    uint32_t ctas;           // of the attention kernel (tree_grid)
    uint32_t prep_heads;     // query heads of one warp of the prep kernel (the launcher's choice)
    uint32_t box_keys;       // keys of one TMA box of K: a power of two, at most 128
    float eps;
    float scale_log2;        // softmax scale * log2(e)
    uint32_t flags;          // SLOTKV_OPT_* norm options
    ScoreRule rule;          // doc_start: [n_req]
};
constexpr uint32_t kTreeSkip = 0xFFFFFFFFu;
// Places of a request that 32-bit arithmetic on them leaves room for (a table may name more).
constexpr uint32_t kTreePlaces = 0x7FFFFF00u;
// A unit to join: its first node and row, rows (0: none), kv head, request, the step from one
// of its CTAs to the next, and their number; and whether the CTA gave up.
constexpr uint32_t kTreeJoin = 8;
// A CTA's plan: what its roles need to know of its first unit (TreeWord) and that unit's
// tiles, then where to go on: size of the sets, block of a set, request, groups of the size
// with one tile more than the others; tiles into the request, tiles left, the part's end,
// tiles of a group (64 bits each).
constexpr uint32_t kTreePlan = 28;
enum TreePlanWord { kPlanUnitTiles = 12, kPlanSize, kPlanMember, kPlanReq, kPlanOver, kPlanOff = 18, kPlanLeft = 20,
                    kPlanEnd = 22, kPlanEach = 24 };
enum TreeJoinWord { kJoinTok, kJoinRow0, kJoinRows, kJoinKvHead, kJoinReq, kJoinStep, kJoinParts,
                    kJoinGaveUp };

// Rows of a block (a unit of work), and the keys and dims of a piece of V.
__host__ __device__ constexpr uint32_t tree_rows(int hd) { return hd == 256 ? 32u : 64u; }
__host__ __device__ constexpr uint32_t tree_v_dims(int hd) { return hd < 128 ? hd : 128u; }
__host__ __device__ constexpr uint32_t tree_v_keys(int hd) { return 4096u / tree_v_dims(hd); }
// CTAs of the attention kernel: one per SM, and enough for a group of each size.
inline uint32_t tree_grid(uint32_t sms) { return sms < 15u ? 15u : sms; }
// Head rows of partial results that a call can leave.
inline size_t tree_partial_rows(int hd, uint32_t sms) { return (size_t)2 * tree_grid(sms) * tree_rows(hd); }

// Enqueue the kernels of a call (prep, attention, combine); tmK:
// the 128-byte-swizzled view of K with boxes of 32 floats x box_keys rows, tmV:
// V's with boxes of tree_v_dims(hd) floats x min(box_keys, tree_v_keys(hd))
// rows, not swizzled.  Return a cudaError_t value.
int launch_tree_hd64(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, uint32_t sms,
                     cudaStream_t stream);
int launch_tree_hd128(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, uint32_t sms,
                      cudaStream_t stream);
int launch_tree_hd256(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, uint32_t sms,
                      cudaStream_t stream);

}  // namespace slotkv
