// maps.cu -- request lengths turned into the index arrays of a step, on the
// device: slot_kv_token_map (one slot and position per prompt token, what a
// batched prefill takes) and slot_kv_extend_tables (block tables extended
// from a free list, what a paged decode takes).
//
// Both are an exclusive prefix sum of one count per request, then one output
// per counted unit (a token, a block).  They move a few KB to a few MB, so a
// call is bound by latency: each is one kernel with no second pass and no
// hand-over between CTAs.  A CTA writes the outputs of one tile of
// consecutive units.  It sums all the counts itself -- R loads from L2 spread
// over its threads, each thread a contiguous part of the requests, which up
// to tens of thousands of requests costs less than another kernel or a wait
// for other CTAs would -- and the threads whose part reaches into the tile
// mark, in shared memory, the unit at which each request starts.  A running
// maximum over the marks then tells every unit its request.  Both
// kernels are launched as programmatic dependents, wait for what precedes
// them before anything else, and let their own dependents launch: the set-up
// of one call overlaps the call before it.  Measured back to back: 5 requests
// 2.7 us, 601 requests with 65 thousand tokens 3.5 us, a step of 67 requests'
// tables 3.4 us, the tables of 4099 prompts 8.7 us (a chain of passes: counts,
// scan, marks, owners, free list; one or four CTAs per SM differ by 1 us).
#include <cuda_runtime.h>
#include <stdint.h>

#include "maps.h"

namespace slotkv {
namespace {

constexpr uint32_t kRange = 1u;  // SLOTKV_DEV_RANGE
constexpr int kMapThreads = 512;
constexpr int kMapWarps = kMapThreads / 32;
constexpr uint32_t kMapTile = 2 * kMapThreads;  // units per tile

__device__ __forceinline__ void begin_dependent() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Exclusive prefix sum of one value per thread over the CTA; total: its sum.
__device__ uint64_t block_exclusive(uint64_t v, uint64_t* warp_sums, uint64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kMapWarps; ++w) {
        const uint64_t x = warp_sums[w];
        before += w < warp ? x : 0u;
        all += x;
    }
    total = all;
    return before + incl - v;
}

// This thread's contiguous part [r0, r1) of the R requests.
__device__ __forceinline__ void my_part(uint32_t R, uint32_t& r0, uint32_t& r1) {
    const uint32_t per = (R + kMapThreads - 1) / kMapThreads;  // R < 2^31
    const uint32_t a = threadIdx.x * per;
    r0 = a < R ? a : R;
    r1 = r0 + per < R ? r0 + per : R;
}

// mark[i] = i + 1 where a request starts at the tile's unit i, else 0; on
// return the unit at which the request of each unit starts, plus 1 (0: no
// request covers it).
__device__ void tile_owners(uint32_t* mark, uint32_t* warp_max) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t a = mark[2 * threadIdx.x], b = mark[2 * threadIdx.x + 1];
    uint32_t m = a > b ? a : b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, m, off);
        if (lane >= off) m = m > o ? m : o;
    }
    if (lane == 31) warp_max[warp] = m;
    uint32_t before = __shfl_up_sync(0xffffffffu, m, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before = before > warp_max[w] ? before : warp_max[w];
    const uint32_t first = before > a ? before : a;
    mark[2 * threadIdx.x] = first;
    mark[2 * threadIdx.x + 1] = first > b ? first : b;
    __syncthreads();
}

// One tile of tokens per CTA; CTA 0 also writes the starts and checks the
// requests.
__global__ void __launch_bounds__(kMapThreads) slotkv_token_map_kernel(const TokenMapParams P) {
    __shared__ uint64_t sums[kMapWarps];
    __shared__ uint32_t warp_max[kMapWarps];
    __shared__ uint32_t mark[kMapTile], slot_at[kMapTile], pos_at[kMapTile];
    begin_dependent();
    const uint64_t t0 = static_cast<uint64_t>(blockIdx.x) * kMapTile;
    mark[threadIdx.x] = mark[threadIdx.x + kMapThreads] = 0;
    uint32_t r0, r1;
    my_part(P.R, r0, r1);
    uint64_t sum = 0, total;
#pragma unroll 8
    for (uint32_t r = r0; r < r1; ++r) sum += __ldg(P.fresh + r);
    uint64_t at = block_exclusive(sum, sums, total);
    const bool head = blockIdx.x == 0;
    if (head || (at < t0 + kMapTile && at + sum > t0)) {
        for (uint32_t r = r0; r < r1; ++r) {
            const uint32_t n = __ldg(P.fresh + r);
            const bool here = n && at < t0 + kMapTile && at + n > t0;
            if (head || here) {
                const uint32_t slot = __ldg(P.slots + r), past = __ldg(P.past + r);
                const bool ok = slot < P.n_slots && static_cast<uint64_t>(past) + n <= P.slot_ctx;
                if (head) {
                    P.starts[r] = at < 0xFFFFFFFFull ? static_cast<uint32_t>(at) : 0xFFFFFFFFu;
                    if (n && !ok) atomicOr(P.status, kRange);
                }
                if (here) {
                    const uint32_t i = at > t0 ? static_cast<uint32_t>(at - t0) : 0u;
                    mark[i] = i + 1;
                    slot_at[i] = ok ? slot : 0xFFFFFFFFu;
                    pos_at[i] = past + (at < t0 ? static_cast<uint32_t>(t0 - at) : 0u);
                }
            }
            at += n;
        }
    }
    if (head && threadIdx.x == 0) {
        P.starts[P.R] = total < 0xFFFFFFFFull ? static_cast<uint32_t>(total) : 0xFFFFFFFFu;
        if (total > P.n_tok) atomicOr(P.status, kRange);
    }
    __syncthreads();
    tile_owners(mark, warp_max);
    const uint64_t end = total < P.n_tok ? total : P.n_tok;
#pragma unroll
    for (uint32_t k = 0; k < 2; ++k) {
        const uint32_t i = threadIdx.x + k * kMapThreads;
        if (t0 + i < end) {
            const uint32_t j = mark[i] - 1;
            P.tok_slots[t0 + i] = slot_at[j];
            P.tok_positions[t0 + i] = pos_at[j] + (i - j);
        }
    }
}

// Blocks request r needs beyond the ones it has; have: those; false for a
// request whose blocks would not fit in its table.
__device__ __forceinline__ bool blocks_needed(const ExtendTablesParams& P, uint32_t r,
                                              uint32_t& have, uint32_t& need) {
    const uint32_t past = __ldg(P.past + r), fresh = __ldg(P.fresh + r);
    const uint64_t len = static_cast<uint64_t>(past) + fresh;
    // blocks of n keys, rounded up (the divisions are most of the kernel's
    // instructions, so a power of two shifts)
    auto blocks = [&](uint32_t n) {
        return n ? (P.shift < 32u ? (n - 1u) >> P.shift : (n - 1u) / P.block) + 1u : 0u;
    };
    have = blocks(past);
    need = 0;
    if (len > 0xFFFFFFFFull) return false;
    const uint32_t want = blocks(static_cast<uint32_t>(len));
    if (want > P.bt_stride) return false;
    need = want - have;
    return true;
}

// Tiles of new blocks, one after the other over the grid.  The grid's last CTA,
// which has the fewest of them, checks the requests and finds the new head.
// It writes it at once, unless that is the word the other CTAs may still have
// to read the old one from: then the last CTA to finish does (1.5 us more).
__global__ void __launch_bounds__(kMapThreads)
    slotkv_extend_tables_kernel(const ExtendTablesParams P) {
    __shared__ uint64_t sums[kMapWarps];
    __shared__ uint32_t warp_max[kMapWarps];
    __shared__ uint32_t mark[kMapTile];
    __shared__ uint64_t entry_at[kMapTile];  // table entry of the marked unit
    __shared__ uint32_t used;
    begin_dependent();
    const uint32_t head = __ldcg(P.head);
    const uint64_t avail = head < P.n_free ? P.n_free - head : 0u;
    uint32_t r0, r1;
    my_part(P.R, r0, r1);
    if (threadIdx.x == 0) used = 0;
    uint64_t sum = 0, total;
#pragma unroll 4
    for (uint32_t r = r0; r < r1; ++r) {
        uint32_t have, need;
        blocks_needed(P, r, have, need);
        sum += need;
    }
    const uint64_t at0 = block_exclusive(sum, sums, total);
    const bool same_word = P.head_out == P.head && gridDim.x > 1;
    if (blockIdx.x == gridDim.x - 1) {
        uint64_t at = at0;
        uint32_t last = 0;
#pragma unroll 4
        for (uint32_t r = r0; r < r1; ++r) {
            uint32_t have, need;
            const bool ok = blocks_needed(P, r, have, need);
            at += need;
            if (!ok || (need && at > avail)) atomicOr(P.status, kRange);
            if (need && at <= avail) last = static_cast<uint32_t>(at);
        }
        if (last) atomicMax(&used, last);
        __syncthreads();
        if (threadIdx.x == 0) *(same_word ? P.scratch + 1 : P.head_out) = head + used;
    }
    const uint64_t end = total < avail ? total : avail;
    for (uint64_t t0 = static_cast<uint64_t>(blockIdx.x) * kMapTile; t0 < end;
         t0 += static_cast<uint64_t>(gridDim.x) * kMapTile) {
        mark[threadIdx.x] = mark[threadIdx.x + kMapThreads] = 0;
        __syncthreads();
        if (at0 < t0 + kMapTile && at0 + sum > t0) {
            uint64_t at = at0;
            for (uint32_t r = r0; r < r1; ++r) {
                uint32_t have, need;
                blocks_needed(P, r, have, need);
                // (a request that the free list cannot serve whole is marked
                // too, with no table entry)
                if (need && at < t0 + kMapTile && at + need > t0) {
                    const uint32_t i = at > t0 ? static_cast<uint32_t>(at - t0) : 0u;
                    const uint64_t entry = static_cast<uint64_t>(r) * P.bt_stride + have +
                                           (at < t0 ? t0 - at : 0u);
                    mark[i] = i + 1;
                    entry_at[i] = at + need <= avail ? entry : ~0ull;
                }
                at += need;
            }
        }
        __syncthreads();
        tile_owners(mark, warp_max);
#pragma unroll
        for (uint32_t k = 0; k < 2; ++k) {
            const uint32_t i = threadIdx.x + k * kMapThreads;
            if (t0 + i < end) {
                const uint32_t j = mark[i] - 1;
                if (entry_at[j] != ~0ull)
                    P.block_tables[entry_at[j] + (i - j)] = __ldg(P.free_blocks + head + t0 + i);
            }
        }
        __syncthreads();  // the marks are free again
    }
    if (!same_word) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(P.scratch, 1u) == gridDim.x - 1) {
            __threadfence();
            *P.head_out = __ldcg(P.scratch + 1);
            P.scratch[0] = 0;
        }
    }
}

}  // namespace

template <typename P>
static int launch_dependent(void (*kernel)(const P), unsigned ctas, const P& p,
                            cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kMapThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p));
}

int launch_token_map(const TokenMapParams& p, cudaStream_t stream) {
    const uint32_t tiles = p.n_tok ? (p.n_tok - 1) / kMapTile + 1 : 1;
    return launch_dependent(slotkv_token_map_kernel, tiles, p, stream);
}

int launch_extend_tables(const ExtendTablesParams& p, uint32_t sms, cudaStream_t stream) {
    // no more tiles than the free list or the tables have entries
    const uint64_t room = static_cast<uint64_t>(p.R) * p.bt_stride;
    const uint64_t most = room < p.n_free ? room : p.n_free;
    const uint64_t tiles = most ? (most - 1) / kMapTile + 1 : 1;
    // (four CTAs of 512 threads fit on an SM)
    const uint64_t ctas = tiles < 4ull * sms ? tiles : 4ull * sms;
    return launch_dependent(slotkv_extend_tables_kernel, static_cast<unsigned>(ctas), p, stream);
}

}  // namespace slotkv
