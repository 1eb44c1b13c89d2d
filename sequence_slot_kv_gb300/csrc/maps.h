// maps.h -- launch parameters of the request-length kernels (maps.cu).
// Plain data only.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace slotkv {

struct TokenMapParams {
    const uint32_t* slots;  // [R]
    const uint32_t* past;   // [R]
    const uint32_t* fresh;  // [R]
    uint32_t* starts;       // [R + 1]
    uint32_t* tok_slots;    // [n_tok]
    uint32_t* tok_positions;
    uint32_t* status;       // sticky SLOTKV_DEV_* flags
    uint32_t R, n_tok, n_slots, slot_ctx;
};

struct ExtendTablesParams {
    const uint32_t* past;         // [R]
    const uint32_t* fresh;        // [R]
    uint32_t* block_tables;       // [R][bt_stride]
    const uint32_t* free_blocks;  // [n_free]
    const uint32_t* head;         // [1]
    uint32_t* head_out;           // [1], may be head
    uint32_t* scratch;            // handle-owned: [0] CTAs done (0 between calls), [1] new head
    uint32_t* status;
    uint32_t R, bt_stride, block, n_free;
    uint32_t shift;               // log2(block), or 32 where block is no power of two
};

// Enqueue one kernel each; return a cudaError_t value.
int launch_token_map(const TokenMapParams& p, cudaStream_t stream);
int launch_extend_tables(const ExtendTablesParams& p, uint32_t sms, cudaStream_t stream);

}  // namespace slotkv
