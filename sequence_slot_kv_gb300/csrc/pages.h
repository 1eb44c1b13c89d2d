// pages.h -- launch parameters of the kernels that move, share and give back
// cache rows and pool blocks (pages.cu).  Plain data only.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace slotkv {

// A handle's K and V as a pool of n_blocks blocks of `block` positions.
struct PoolView {
    float* K;
    float* V;
    uint32_t n_blocks, block, kv_dim;
    uint32_t* status;  // sticky SLOTKV_DEV_* flags
};

struct KeepPathParams {
    PoolView pool;                 // slots: n_slots blocks of slot_ctx positions
    const uint32_t* slots;         // [R], or null: paged
    const uint32_t* block_tables;  // [R][bt_stride]
    const uint32_t* past;          // [R]
    const uint32_t* starts;        // [R + 1]
    const uint32_t* n_keep;        // [R]
    const uint32_t* path;          // [n_tok]
    uint32_t R, n_tok, bt_stride;
};

struct ForkTablesParams {
    PoolView pool;
    const uint32_t* src;           // [n_fork]
    const uint32_t* past;          // [n_rows]
    const uint32_t* block_tables;  // [n_rows][bt_stride]
    uint32_t* out_tables;          // [n_fork][bt_stride]
    uint32_t* shares;              // [n_blocks]
    const uint32_t* free_blocks;   // [n_free]
    const uint32_t* head;          // [1]
    uint32_t* head_out;            // [1], may be head
    uint32_t* scratch;             // handle-owned: [0] CTAs done (0 between calls), [1] new head
    uint32_t* counts;              // handle-owned: one per kForkRun forks
    uint32_t n_fork, n_rows, bt_stride, n_free;
};
constexpr uint32_t kForkRun = 1024;  // forks that are counted together

struct FreeTablesParams {
    PoolView pool;
    const uint32_t* past;          // [R]
    const uint32_t* keep;          // [R], or null: 0
    const uint32_t* block_tables;  // [R][bt_stride]
    uint32_t* shares;              // [n_blocks], or null
    uint32_t* free_blocks;         // [n_free]
    const uint32_t* head;          // [1]
    uint32_t* head_out;            // [1], may be head
    uint32_t* counts;              // handle-owned: [kFreeCtas + 1]
    uint32_t R, bt_stride, n_free;
};
constexpr uint32_t kFreeCtas = 1024;  // at most, of the kernels that free many entries

struct CompactPoolParams {
    PoolView pool;
    const uint32_t* past;          // [R]
    uint32_t* block_tables;        // [R][bt_stride]
    uint32_t* shares;              // [n_blocks], or null
    uint32_t* free_blocks;         // [n_free]
    uint32_t* head;                // [1]
    uint32_t* scratch;             // handle-owned: compact_scratch_words(n_blocks)
    uint32_t R, bt_stride, n_free;
};

// map of new ids, the blocks that move, where they go, [0] blocks in use, [1] moves
inline size_t compact_scratch_words(uint32_t n_blocks) { return 3 * (size_t)n_blocks + 4; }

// Nodes a request's tree may have.
constexpr uint32_t kMaxTree = 256;

// Enqueue the kernels of a call; return a cudaError_t value.
int launch_keep_path(const KeepPathParams& p, cudaStream_t stream);
int launch_fork_tables(const ForkTablesParams& p, uint32_t sms, cudaStream_t stream);
int launch_free_tables(const FreeTablesParams& p, uint32_t sms, cudaStream_t stream);
int launch_compact_pool(const CompactPoolParams& p, uint32_t sms, cudaStream_t stream);

}  // namespace slotkv
