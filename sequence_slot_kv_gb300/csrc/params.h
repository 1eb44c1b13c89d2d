// params.h -- launch parameters shared by the host side and the kernels of
// libslotkv.  Plain data only.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include <type_traits>

namespace slotkv {

struct DecodeParams {
    const float* q;          // [B][n_head][hd]
    const float* k_new;      // [B][n_kv_head][hd]
    const float* v_new;      // [B][n_kv_head][hd]
    const uint32_t* positions;
    const uint32_t* slots;
    const float* q_norm_w;   // [hd]
    const float* k_norm_w;   // [hd]
    const float* inv_freq;   // [hd/2]
    const float* sinks;      // [n_head] or null
    float* out;              // [B][n_head][hd]
    float* K;                // slot buffers [n_slots][slot_ctx][n_kv_head][hd]
    float* V;
    float* ws_ml;            // split partials (m, l): [rows][n_head][max_splits][2]
    float* ws_acc;           // split partials acc:    [rows][n_head][max_splits][hd]
    uint32_t* counters;      // finished-split counters: [rows][n_kv_head]
    uint32_t* items;         // work list: [rows * n_kv_head * max_splits][4] records
                             // (packed item, position, tensor row of key p, 0)
    uint32_t* plan;          // [0] items in the list, [1] next item to hand out
    uint32_t* status;        // sticky SLOTKV_DEV_* flags
    uint32_t n_slots, slot_ctx, n_head, n_kv_head, B;
    uint32_t chunk_min;      // split policy, see split_chunk()
    uint32_t max_splits;
    float eps;
    float scale_log2;        // softmax scale * log2(e): scores live in base 2
    uint32_t flags;          // SLOTKV_OPT_* norm options
    uint32_t prefill;        // 1: rows are prefill tokens (keys all read from the slot)
    // Paged mode (block_tables non-null): K and V are a pool of n_slots blocks
    // of slot_ctx positions and row b's key t lives in block
    // block_tables[b * bt_stride + t / slot_ctx] at offset t % slot_ctx;
    // slot_ctx is then a multiple of the tile height.  slots is unused.
    const uint32_t* block_tables = nullptr;
    uint32_t bt_stride = 0;
    // Static first items: decode CTA c < static_items starts with
    // split 0 of (row c / n_kv_head, kv head c % n_kv_head) without waiting for
    // the plan, which leaves those items out of its list.  0: none.
    uint32_t static_items = 0;
    // Static second items (only when static_items covers every pair): decode
    // CTA static_items + q, q < static_second, starts with split 1 of pair q
    // if that row has a second split, and the plan leaves those items out of
    // its list too.  0: none.
    uint32_t static_second = 0;
    // 1: every item is a static first item (no more (row, kv head) pairs than
    // CTAs, one split each): no plan kernel runs, its list is empty, and the
    // decode kernel is launched in plain stream order.
    uint32_t no_plan = 0;
};

// The tensor-core prefill (head dims 64 and 128): prep, plan and attention
// kernels over tiles of consecutive same-slot tokens (see prefill_tc.cuh).
struct PrefillParams {
    const float* q;          // [n_tok][n_head][hd]
    const float* k_new;      // [n_tok][n_kv_head][hd]
    const float* v_new;      // [n_tok][n_kv_head][hd]
    const uint32_t* positions;
    const uint32_t* slots;
    const float* q_norm_w;
    const float* k_norm_w;
    const float* inv_freq;
    const float* sinks;      // [n_head] or null
    float* out;              // [n_tok][n_head][hd]
    float* K;                // slot buffers [n_slots][slot_ctx][n_kv_head][hd]
    float* V;
    float* q_rot;            // workspace [n_tok][n_head][hd]: normed, rotated, scaled q
    uint32_t* tiles;         // workspace [n_tok][4]: first token, tokens, slot, largest position
    uint32_t* tile_of;       // workspace [n_tok]: each token's tile, then the tiles' hand-out order
    uint32_t* plan;          // [0] items (tiles * n_kv_head), [1] next item to hand out,
                             // [2] scored calls: 1 if the tiles were split
    uint32_t* status;        // sticky SLOTKV_DEV_* flags
    uint32_t n_slots, slot_ctx, n_head, n_kv_head, n_tok;
    float eps;
    float scale_log2;        // softmax scale * log2(e)
    uint32_t flags;          // SLOTKV_OPT_* norm options
};

// The score rule of a scored call (include/slotkv.h, slotkv_scores), in the
// kernels' base-2 units: a score s is log2(e) times the natural one, so the
// cap reads c tanh(s_nat / c) log2(e) = cap_out * tanh(s * cap_in).
struct ScoreRule {
    float cap_in = 0.f, cap_out = 0.f;      // ln 2 / c, c log2(e); cap_out 0: no cap
    uint32_t window = 0;                    // keys t with p - t < window; 0: all
    const float* slopes = nullptr;          // [n_head], natural units, or null
    const uint32_t* doc_start = nullptr;    // [rows]: first key of the row's document, or null
    const uint32_t* prefix_end = nullptr;   // [rows]: keys below it are attended whatever the
                                            // row's position (prefill only), or null
};

// The rows of a shared call: row b's positions 0 .. lens[b] - 1 live in slot
// slots[b] of another handle's buffers (n_slots slots of slot_ctx positions),
// the rest in its own slot from position 0 on.  lens null: not a shared call.
struct SharedRows {
    const uint32_t* slots = nullptr;
    const uint32_t* lens = nullptr;
    uint32_t n_slots = 0, slot_ctx = 0;
};

// What the prefix pass of a shared call leaves for the decode kernel, and the
// splits of a scored prefill for its combine kernel.  rec[b] = (first partial
// row, stride, splits, 0), then the row's position and the first and last key
// it attends, for the attention kernel: split s of row b, head h, is partial
// (rec.x + s * rec.y) * n_head + h, (m, l) and an unnormalised accumulator.
struct Partials {
    uint32_t* rec = nullptr;  // [rows][8]
    float* ml = nullptr;      // [partials][2]
    float* acc = nullptr;     // [partials][hd]
};

struct ScoredDecodeParams : DecodeParams {
    ScoreRule rule;
    SharedRows shared;
    Partials part;
};

struct ScoredPrefillParams : PrefillParams {
    ScoreRule rule;
    SharedRows shared;       // shared call: K, V, n_slots and slot_ctx are the prefix handle's,
                             // own_* the rows' own slots and their geometry
    const uint32_t* own_slots = nullptr;
    uint32_t own_n_slots = 0, own_ctx = 0;
    Partials part;
    uint32_t* tile_lo = nullptr;  // workspace [n_tok]: each tile's smallest key
    // workspace [n_tok + splits][8], an entry per (tile, split): first token,
    // tokens, row of the first key in the [rows][kv_dim] view, first key; keys,
    // split, 0, 0
    uint32_t* list = nullptr;
    uint32_t sms = 0;             // SMs (= the attention kernel's CTAs)
    uint32_t after_plan = 0;      // 1: a decode plan kernel precedes on the stream
};

template <bool SC>
using decode_params_t = std::conditional_t<SC, ScoredDecodeParams, DecodeParams>;
template <bool SC>
using prefill_params_t = std::conditional_t<SC, ScoredPrefillParams, PrefillParams>;

// Keys per split chunk for a row with n_keys keys (p + 1).  Depends only on
// n_keys and the geometry so that a row's result never depends on the batch.
__host__ __device__ inline uint32_t split_chunk(uint32_t n_keys, uint32_t chunk_min,
                                                uint32_t max_splits, uint32_t tile) {
    uint32_t per = (n_keys + max_splits - 1) / max_splits;
    per = (per + tile - 1) / tile * tile;
    return per > chunk_min ? per : chunk_min;
}

// Tile height (keys per pipeline stage) for a head dim: 16 KiB of K + 16 KiB of V.
__host__ __device__ constexpr int tile_keys(int hd) { return 4096 / hd; }

// A work item is one (row, split, kv head), packed as row << 16 | split << 8 |
// kv head; rows <= 65535, splits and kv heads <= 256.
__host__ __device__ inline uint32_t pack_item(uint32_t b, uint32_t split, uint32_t kvh) {
    return (b << 16) | (split << 8) | kvh;
}

// Work-list records the workspace must hold: one per (row, kv head, split);
// each record is 4 u32 (16 bytes).
inline size_t plan_capacity(uint32_t rows, uint32_t n_kv_head, uint32_t max_splits) {
    return (size_t)rows * n_kv_head * max_splits;
}
constexpr int kItemWords = 4;

// Sets the calling thread's slot_kv_last_error() message.
void set_last_error(const char* msg);

// Launchers, one translation unit per head dim.  Each enqueues the plan kernel
// and then the persistent decode kernel on `stream` with `ctas` CTAs.  Return a
// cudaError_t value.
int launch_decode_hd64(int G, const DecodeParams& p, const CUtensorMap& tmK,
                       const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream);
int launch_decode_hd128(int G, const DecodeParams& p, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream);
int launch_decode_hd256(int G, const DecodeParams& p, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream);

// The small-call decode kernel (one CTA per (row, kv head), see
// decode_small.cuh): taken when a decode call has at most two CTAs' worth
// of (row, kv head) pairs per SM and slots of at most small_max_keys keys.
int launch_small_hd64(int G, const DecodeParams& p, cudaStream_t stream);
int launch_small_hd128(int G, const DecodeParams& p, cudaStream_t stream);
int launch_small_hd256(int G, const DecodeParams& p, cudaStream_t stream);
__host__ __device__ constexpr int small_max_keys(int hd) { return 8 * tile_keys(hd); }

// Tensor-core prefill launchers (prep, plan, attention on `stream`); tmK and
// tmV are the 128-byte-swizzled views of the slot buffers with a box of 32
// floats x prefill_tile_keys(hd) rows.  Return a cudaError_t value.
int launch_prefill_tc_hd64(int G, const PrefillParams& p, const CUtensorMap& tmK,
                           const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream);
int launch_prefill_tc_hd128(int G, const PrefillParams& p, const CUtensorMap& tmK,
                            const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream);

// The scored forms (capped scores, distance bias, masks; see score_rule.cuh)
// of the three kinds above, and the prefix pass of a shared decode call
// (plan, q preparation, attention into partials).  A shared decode call is
// launched in two parts around its prefix pass, first the decode plan (if
// its shape has one), then the attention, a programmatic dependent of the pass.
enum class ScoredPart { whole, plan, attention };
int launch_scored_hd64(int G, const ScoredDecodeParams& p, const CUtensorMap& tmK,
                       const CUtensorMap& tmV, unsigned ctas, bool small, ScoredPart part,
                       cudaStream_t stream);
int launch_scored_hd128(int G, const ScoredDecodeParams& p, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, unsigned ctas, bool small, ScoredPart part,
                       cudaStream_t stream);
int launch_scored_hd256(int G, const ScoredDecodeParams& p, const CUtensorMap& tmK,
                        const CUtensorMap& tmV, unsigned ctas, bool small, ScoredPart part,
                       cudaStream_t stream);
int launch_scored_prefill_hd64(int G, const ScoredPrefillParams& p, const CUtensorMap& tmK,
                               const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream);
int launch_scored_prefill_hd128(int G, const ScoredPrefillParams& p, const CUtensorMap& tmK,
                                const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream);

// (tile, split) items per SM and kv head that the scored prefill's plan may
// make by splitting; a call with more tiles than kSplitBelow items per SM is
// never split.
constexpr uint32_t kSplitBelow = 2, kSplitMost = 8, kMaxSplits = 64;
// head rows of partials that splits can need, however many rows a call has: 128
// query rows per split item
inline size_t partial_head_rows(uint32_t sms) { return (size_t)128 * kSplitMost * sms; }

// Keys per pipeline stage of the tensor-core prefill.
__host__ __device__ constexpr int prefill_tile_keys(int hd, bool scored = false) {
    return scored && hd == 128 ? 32 : 64;
}

}  // namespace slotkv
