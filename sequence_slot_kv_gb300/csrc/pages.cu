// pages.cu -- cache rows and pool blocks moved, shared and given back, on the
// device: slot_kv_keep_path (the rows of a verified tree's accepted path),
// slot_kv_fork_tables (tables that share full blocks and copy the partial
// one), slot_kv_free_tables (blocks back on the free list) and
// slot_kv_compact_pool (the blocks in use moved to the pool's front).
//
// All of them move bytes and count; there is no arithmetic to speak of.  Small
// calls are bound by their dependent loads (a few round trips to L2), large
// ones by the rows they copy.
#include <cuda_runtime.h>
#include <stdint.h>

#include "pages.h"

namespace slotkv {
namespace {

constexpr uint32_t kRange = 1u;  // SLOTKV_DEV_RANGE
constexpr int kCopyThreads = 256;
constexpr uint32_t kBatch = 8;   // 16-byte pieces a thread has in flight
constexpr uint32_t kMaxPlaces = 0x7FFFFF00u;  // places of a request (a table may name more)

__device__ __forceinline__ void begin_dependent() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ uint32_t blocks_of(uint32_t keys, uint32_t block) {
    return keys ? (keys - 1u) / block + 1u : 0u;
}

// n float4s from src to dst, by the threads i0, i0 + step, ...; the ranges do
// not overlap.
__device__ __forceinline__ void copy_float4(const float4* __restrict__ src,
                                            float4* __restrict__ dst, uint64_t n, uint32_t i0,
                                            uint32_t step) {
    for (uint64_t i = i0; i < n; i += static_cast<uint64_t>(kBatch) * step) {
        float4 x[kBatch];
#pragma unroll
        for (uint32_t k = 0; k < kBatch; ++k) {
            const uint64_t j = i + static_cast<uint64_t>(k) * step;
            if (j < n) x[k] = __ldcs(src + j);
        }
#pragma unroll
        for (uint32_t k = 0; k < kBatch; ++k) {
            const uint64_t j = i + static_cast<uint64_t>(k) * step;
            if (j < n) dst[j] = x[k];
        }
    }
}

// ------------------------------------------------------------------ keep path
// Row past + k of the request takes row past + path[k], k in order.  path is
// strictly increasing, so path[k] >= k: row k is written after every row that
// it was the source of has been read.  A thread owns one 16-byte column of the
// request's rows and goes through the path in order, eight loads before their
// eight stores, so no thread waits for another and the moves may overlap.
// A request whose table names a block outside the pool, anywhere up to its last
// node, moves nothing, as the tree call attends nothing of it.
// Bound by the launch and three dependent loads: 3 requests 2.7 us, 193 requests
// that move 9.2 MB 4.9.
__global__ void __launch_bounds__(kCopyThreads) slotkv_keep_path_kernel(const KeepPathParams P) {
    __shared__ uint32_t from[kMaxTree], to[kMaxTree];
    begin_dependent();
    const uint32_t r = blockIdx.x;
    const uint32_t s0 = __ldg(P.starts + r), s1 = __ldg(P.starts + r + 1);
    const uint32_t n = __ldg(P.n_keep + r), past = __ldg(P.past + r);
    if (n == 0) return;
    uint64_t limit = P.slots ? P.pool.block : static_cast<uint64_t>(P.bt_stride) * P.pool.block;
    limit = limit < kMaxPlaces ? limit : kMaxPlaces;
    bool ok = s0 <= s1 && s1 <= P.n_tok && s1 - s0 <= kMaxTree && n <= s1 - s0 &&
              static_cast<uint64_t>(past) + (s1 - s0) <= limit;
    const uint32_t slot = P.slots ? __ldg(P.slots + r) : 0u;
    if (P.slots) ok = ok && slot < P.pool.n_blocks;
    // (a thread's first entry of the table is on its way while the path is looked at)
    const uint32_t* row = P.slots ? nullptr : P.block_tables + static_cast<size_t>(r) * P.bt_stride;
    const uint32_t used = ok && row ? (past + (s1 - s0) - 1) / P.pool.block + 1 : 0u;
    const uint32_t first = threadIdx.x < used ? __ldg(row + threadIdx.x) : 0u;
    // row of the request's position p in the [rows][kv_dim] view
    auto row_of = [&](uint32_t p) {
        if (P.slots) return slot * P.pool.block + p;
        return __ldg(row + p / P.pool.block) * P.pool.block + p % P.pool.block;
    };
    if (ok) {
        for (uint32_t k = threadIdx.x; k < n; k += kCopyThreads) {
            const uint32_t i = __ldg(P.path + s0 + k);
            const uint32_t before = k ? __ldg(P.path + s0 + k - 1) : 0u;
            if (i >= s1 - s0 || (k && i <= before)) {
                ok = false;
            } else {
                from[k] = row_of(past + i);
                to[k] = row_of(past + k);
            }
        }
    }
    ok = ok && first < P.pool.n_blocks;
#pragma unroll 4
    for (uint32_t e = threadIdx.x + kCopyThreads; e < used; e += kCopyThreads)
        ok = __ldg(row + e) < P.pool.n_blocks && ok;
    if (!__syncthreads_and(ok)) {
        if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(P.pool.status, kRange);
        return;
    }
    const uint32_t cols = P.pool.kv_dim / 4;
    for (uint32_t c = blockIdx.y * kCopyThreads + threadIdx.x; c < 2 * cols;
         c += gridDim.y * kCopyThreads) {
        float4* X = reinterpret_cast<float4*>(c < cols ? P.pool.K : P.pool.V) +
                    (c < cols ? c : c - cols);
        for (uint32_t k0 = 0; k0 < n; k0 += kBatch) {
            float4 x[kBatch];
#pragma unroll
            for (uint32_t k = 0; k < kBatch; ++k)
                if (k0 + k < n && from[k0 + k] != to[k0 + k])
                    x[k] = X[static_cast<size_t>(from[k0 + k]) * cols];
#pragma unroll
            for (uint32_t k = 0; k < kBatch; ++k)
                if (k0 + k < n && from[k0 + k] != to[k0 + k])
                    X[static_cast<size_t>(to[k0 + k]) * cols] = x[k];
        }
    }
}

// ------------------------------------------------------------------ fork
// Whether fork j takes a block of the free list; false in ok: out of range.
__device__ __forceinline__ bool fork_needs(const ForkTablesParams& P, uint32_t j, bool& ok,
                                           uint32_t& s, uint32_t& past) {
    s = __ldg(P.src + j);
    ok = s < P.n_rows;
    past = ok ? __ldg(P.past + s) : 0u;
    ok = ok && blocks_of(past, P.pool.block) <= P.bt_stride;
    return ok && past % P.pool.block != 0u;
}

// The forks of each run of kForkRun that take a block, for calls of more than kForkOne.
__global__ void __launch_bounds__(kCopyThreads) slotkv_fork_count_kernel(const ForkTablesParams P) {
    __shared__ uint32_t count;
    begin_dependent();
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    const uint32_t j0 = blockIdx.x * kForkRun, j1 = P.n_fork - j0 < kForkRun ? P.n_fork : j0 + kForkRun;
    uint32_t n = 0;
    for (uint32_t j = j0 + threadIdx.x; j < j1; j += kCopyThreads) {
        bool ok;
        uint32_t s, past;
        n += fork_needs(P, j, ok, s, past);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0 && n) atomicAdd(&count, n);
    __syncthreads();
    if (threadIdx.x == 0) P.counts[blockIdx.x] = count;
}

// CTA (fork, part): counts the forks before its own that take a block, which
// names its own; part 0 writes the fork's table, and every part copies its
// share of the partial block.  Every CTA reads the lengths of the forks before it,
// so that nothing waits: one kernel, and partial blocks at the copy's rate (192 MB in
// 30 us, 6.4 TB/s; what a call of few rows takes is its four dependent loads).
// With RUNS it reads those before it in its run, and the counts of the runs before that.
template <bool RUNS>
__global__ void __launch_bounds__(kCopyThreads) slotkv_fork_tables_kernel(const ForkTablesParams P) {
    __shared__ uint32_t count;
    begin_dependent();
    const uint32_t i = blockIdx.x;
    const uint32_t head = __ldcg(P.head);
    const uint32_t avail = head < P.n_free ? P.n_free - head : 0u;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    uint32_t before = 0;
    if (RUNS)
        for (uint32_t c = threadIdx.x; c < i / kForkRun; c += kCopyThreads) before += __ldcg(P.counts + c);
    for (uint32_t j = threadIdx.x + (RUNS ? i / kForkRun * kForkRun : 0u); j < i; j += kCopyThreads) {
        bool ok;
        uint32_t s, past;
        before += fork_needs(P, j, ok, s, past);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if ((threadIdx.x & 31) == 0 && before) atomicAdd(&count, before);
    __syncthreads();
    const uint32_t at = count;  // blocks that the forks before this one take
    bool ok = false;
    uint32_t s = 0, past = 0;
    const bool need = i < P.n_fork && fork_needs(P, i, ok, s, past);
    const bool served = !need || at < avail;
    if (blockIdx.y == 0 && threadIdx.x == 0 && i < P.n_fork && !(ok && served))
        atomicOr(P.pool.status, kRange);
    if (ok && served) {
        const uint32_t full = past / P.pool.block, rest = past % P.pool.block;
        const uint32_t* row = P.block_tables + static_cast<size_t>(s) * P.bt_stride;
        uint32_t* out = P.out_tables + static_cast<size_t>(i) * P.bt_stride;
        if (blockIdx.y == 0) {
            for (uint32_t e = threadIdx.x; e < full; e += kCopyThreads) {
                const uint32_t id = __ldg(row + e);
                out[e] = id;
                if (id < P.pool.n_blocks)
                    atomicAdd(P.shares + id, 1u);
                else
                    atomicOr(P.pool.status, kRange);
            }
        }
        if (need) {
            const uint32_t id = __ldg(P.free_blocks + head + at), old = __ldg(row + full);
            const bool good = id < P.pool.n_blocks && old < P.pool.n_blocks;
            if (blockIdx.y == 0 && threadIdx.x == 0) {
                out[full] = id;
                if (!good) atomicOr(P.pool.status, kRange);
            }
            if (good && id != old) {
                const size_t block4 = static_cast<size_t>(P.pool.block) * (P.pool.kv_dim / 4);
                const uint64_t n = static_cast<uint64_t>(rest) * (P.pool.kv_dim / 4);
                const uint32_t t = blockIdx.y * kCopyThreads + threadIdx.x;
                const uint32_t step = gridDim.y * kCopyThreads;
                copy_float4(reinterpret_cast<const float4*>(P.pool.K) + old * block4,
                            reinterpret_cast<float4*>(P.pool.K) + id * block4, n, t, step);
                copy_float4(reinterpret_cast<const float4*>(P.pool.V) + old * block4,
                            reinterpret_cast<float4*>(P.pool.V) + id * block4, n, t, step);
            }
        }
    }
    // the last fork's CTA knows the new head; where that is the word the others
    // read the old one from, the last CTA to finish writes it
    const bool last = i + 1 >= P.n_fork && blockIdx.y == 0;
    const uint32_t used = at + (need ? 1u : 0u);
    const uint32_t new_head = head + (used < avail ? used : avail);
    if (P.head_out != P.head) {
        if (last && threadIdx.x == 0) *P.head_out = new_head;
        return;
    }
    if (threadIdx.x == 0) {
        if (last) atomicExch(P.scratch + 1, new_head);
        __threadfence();
        if (atomicAdd(P.scratch, 1u) == gridDim.x * gridDim.y - 1) {
            __threadfence();
            *P.head_out = __ldcg(P.scratch + 1);
            P.scratch[0] = 0;
        }
    }
}

// ------------------------------------------------------------------ cluster phases
// The list kernels below go through phases that all CTAs finish before the
// next: one cluster of CTAs, whose barrier orders their global accesses too.
constexpr int kListThreads = 1024, kListWarps = kListThreads / 32;
constexpr uint32_t kListCtas = 8;

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A word of another CTA's shared memory.
__device__ __forceinline__ uint32_t cluster_load(const uint32_t* p, uint32_t cta) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), v;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(cta));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Exclusive prefix sum, over the cluster's warps in order, of one value per
// warp (the same in all its lanes); total: the sum.
struct ListScan {
    uint32_t warp_sum[kListWarps];
    uint32_t cta_sum;
};
__device__ uint32_t cluster_exclusive(uint32_t v, ListScan& sh, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) sh.warp_sum[warp] = v;
    __syncthreads();
    const uint32_t x = sh.warp_sum[lane];  // (kListWarps = 32)
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0u);
    if (threadIdx.x == 0) sh.cta_sum = 0;
    const uint32_t sum = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if (threadIdx.x == 0) sh.cta_sum = sum;
    cluster_barrier();
    uint32_t at = before;
    total = 0;
    for (uint32_t c = 0; c < gridDim.x; ++c) {
        const uint32_t y = cluster_load(&sh.cta_sum, c);
        if (c < blockIdx.x) at += y;
        total += y;
    }
    cluster_barrier();  // (no CTA leaves, or reuses the word, while others read it)
    return at;
}
static_assert(kListWarps == 32, "one lane per warp");

// A warp's items: 32 table entries of one request each, in entry order.
struct EntryItems {
    uint32_t per_row, begin, end;  // items per request; this warp's [begin, end)
};
__device__ __forceinline__ EntryItems my_items(uint32_t R, uint32_t bt_stride) {
    EntryItems it;
    it.per_row = (bt_stride + 31) / 32;
    const uint64_t n = static_cast<uint64_t>(R) * it.per_row;
    const uint32_t warps = gridDim.x * kListWarps;
    const uint64_t per = (n + warps - 1) / warps;
    const uint64_t b = (blockIdx.x * kListWarps + (threadIdx.x >> 5)) * per;
    it.begin = static_cast<uint32_t>(b < n ? b : n);
    it.end = static_cast<uint32_t>(b + per < n ? b + per : n);
    return it;
}

// ------------------------------------------------------------------ free
// The entry of this lane in an item, if it gives up a block.
struct FreeEntry {
    uint32_t id, code;
    bool live;
};
__device__ __forceinline__ FreeEntry free_entry(const FreeTablesParams& P, uint32_t item,
                                                uint32_t per_row, bool flag) {
    const uint32_t r = item / per_row, e = (item % per_row) * 32 + (threadIdx.x & 31);
    const uint32_t n = blocks_of(__ldg(P.past + r), P.pool.block);
    const uint32_t k = P.keep ? blocks_of(__ldg(P.keep + r), P.pool.block) : 0u;
    FreeEntry x;
    x.live = n <= P.bt_stride && e >= k && e < n;
    const uint32_t at = r * P.bt_stride + e;
    x.id = x.live ? __ldg(P.block_tables + at) : 0u;
    x.code = 0x80000000u + at;
    const bool bad = n > P.bt_stride || (x.live && x.id >= P.pool.n_blocks);
    if (flag && __any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0)
        atomicOr(P.pool.status, kRange);
    x.live = x.live && x.id < P.pool.n_blocks;
    return x;
}

// Which blocks go, and in which order, without an order among the threads: (1)
// every entry takes one from its block's share count, which goes below zero
// where nobody is left; (2) the entries of those blocks leave their place in
// the tables there, as the most negative numbers, and the first one stays
// (atomic minimum); (3) the entry that finds its own place is the one that
// gives the block back; a prefix sum over them gives their places in the list.
// Bound by the steps' round trips to L2: one cluster 6 to 10 us, the four kernels 8.5
// for few entries, 11 for 2048 items of 32, 42 for 16384.
__device__ __forceinline__ void free_take(const FreeTablesParams& P, const EntryItems& it) {
#pragma unroll 4
    for (uint32_t i = it.begin; i < it.end; ++i) {
        const FreeEntry x = free_entry(P, i, it.per_row, false);
        if (x.live) atomicSub(P.shares + x.id, 1u);
    }
}
__device__ __forceinline__ void free_sign(const FreeTablesParams& P, const EntryItems& it) {
    int* shares = reinterpret_cast<int*>(P.shares);
#pragma unroll 4
    for (uint32_t i = it.begin; i < it.end; ++i) {
        const FreeEntry x = free_entry(P, i, it.per_row, false);
        if (x.live && __ldcg(shares + x.id) < 0) {
            const int old = atomicMin(shares + x.id, static_cast<int>(x.code));
            if (old < -1 && old >= -(1 << 30)) atomicOr(P.pool.status, kRange);  // given up twice
        }
    }
}
__device__ __forceinline__ bool free_goes(const FreeTablesParams& P, const FreeEntry& x) {
    return x.live && (!P.shares || __ldcg(P.shares + x.id) == x.code);
}
// A lane's entries that give a block back, of a warp's first items (most warps have
// no more): whether, and which.
constexpr uint32_t kKeptItems = 4;
struct FreeKept {
    uint32_t id[kKeptItems];
    bool go[kKeptItems];
};
__device__ __forceinline__ uint32_t free_count(const FreeTablesParams& P, const EntryItems& it, FreeKept& kept) {
    uint32_t n = 0;
    FreeEntry x[kKeptItems];
#pragma unroll
    for (uint32_t k = 0; k < kKeptItems; ++k)  // (the loads of all first)
        x[k] = it.begin + k < it.end ? free_entry(P, it.begin + k, it.per_row, true) : FreeEntry{0u, 0u, false};
#pragma unroll
    for (uint32_t k = 0; k < kKeptItems; ++k) {
        kept.id[k] = x[k].id;
        kept.go[k] = free_goes(P, x[k]);
        n += __popc(__ballot_sync(0xffffffffu, kept.go[k]));
    }
#pragma unroll 4
    for (uint32_t i = it.begin + kKeptItems; i < it.end; ++i)
        n += __popc(__ballot_sync(0xffffffffu, free_goes(P, free_entry(P, i, it.per_row, true))));
    return n;
}
// The list is a stack below head: total ids end where the taken ones began.
__device__ __forceinline__ void free_give(const FreeTablesParams& P, const EntryItems& it, const FreeKept& kept,
                                          uint32_t head, uint32_t at, uint32_t total) {
    const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
    auto give = [&](uint32_t id, bool go) {
        const uint32_t m = __ballot_sync(0xffffffffu, go), k = at + __popc(m & below);
        if (go) {
            if (head + k >= total) P.free_blocks[head + k - total] = id;
            if (P.shares) P.shares[id] = 0;
        }
        at += __popc(m);
    };
#pragma unroll
    for (uint32_t k = 0; k < kKeptItems; ++k) give(kept.id[k], kept.go[k]);
    for (uint32_t i = it.begin + kKeptItems; i < it.end; ++i) {
        const FreeEntry x = free_entry(P, i, it.per_row, false);
        give(x.id, free_goes(P, x));
    }
}
__device__ __forceinline__ void free_head(const FreeTablesParams& P, uint32_t head0, uint32_t head,
                                          uint32_t total) {
    *P.head_out = head > total ? head - total : 0u;
    if (head != head0 || total > head) atomicOr(P.pool.status, kRange);
}

// One CTA, or one cluster of them: the steps one after the other.
__global__ void __launch_bounds__(kListThreads) slotkv_free_tables_kernel(const FreeTablesParams P) {
    __shared__ ListScan scan;
    begin_dependent();
    const EntryItems it = my_items(P.R, P.bt_stride);
    const uint32_t head0 = __ldcg(P.head), head = head0 < P.n_free ? head0 : P.n_free;
    if (P.shares) {
        free_take(P, it);
        cluster_barrier();
        free_sign(P, it);
        cluster_barrier();
    }
    FreeKept kept;
    uint32_t total;
    const uint32_t at = cluster_exclusive(free_count(P, it, kept), scan, total);
    free_give(P, it, kept, head, at, total);
    if (blockIdx.x == 0 && threadIdx.x == 0) free_head(P, head0, head, total);
}

// Many entries: the steps are kernels over the whole GPU, each a programmatic
// dependent of the one before.  A CTA counts the blocks that its entries give
// back, the last step sums what the CTAs before it counted.
constexpr int kFreeThreads = 256, kFreeWarps = kFreeThreads / 32;
__device__ __forceinline__ EntryItems grid_items(const FreeTablesParams& P) {
    EntryItems it;
    it.per_row = (P.bt_stride + 31) / 32;
    const uint64_t n = static_cast<uint64_t>(P.R) * it.per_row;
    const uint64_t warps = static_cast<uint64_t>(gridDim.x) * kFreeWarps, per = (n + warps - 1) / warps;
    const uint64_t b = (static_cast<uint64_t>(blockIdx.x) * kFreeWarps + (threadIdx.x >> 5)) * per;
    it.begin = static_cast<uint32_t>(b < n ? b : n);
    it.end = static_cast<uint32_t>(b + per < n ? b + per : n);
    return it;
}
__global__ void __launch_bounds__(kFreeThreads) slotkv_free_take_kernel(const FreeTablesParams P) {
    begin_dependent();
    free_take(P, grid_items(P));
}
__global__ void __launch_bounds__(kFreeThreads) slotkv_free_sign_kernel(const FreeTablesParams P) {
    begin_dependent();
    free_sign(P, grid_items(P));
}
__global__ void __launch_bounds__(kFreeThreads) slotkv_free_count_kernel(const FreeTablesParams P) {
    __shared__ uint32_t sums[kFreeWarps];
    begin_dependent();
    FreeKept kept;
    const uint32_t n = free_count(P, grid_items(P), kept);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t all = 0;
        for (int w = 0; w < kFreeWarps; ++w) all += sums[w];
        P.counts[blockIdx.x] = all;
        // (head_out may be head: the next step reads it here)
        if (blockIdx.x == 0) P.counts[kFreeCtas] = __ldcg(P.head);
    }
}
__global__ void __launch_bounds__(kFreeThreads) slotkv_free_give_kernel(const FreeTablesParams P) {
    __shared__ uint32_t sums[kFreeWarps], before_sum[kFreeWarps], all_sum[kFreeWarps];
    begin_dependent();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const EntryItems it = grid_items(P);
    const uint32_t head0 = __ldcg(P.counts + kFreeCtas), head = head0 < P.n_free ? head0 : P.n_free;
    FreeKept kept;
    const uint32_t mine = free_count(P, it, kept);
    uint32_t before = 0, all = 0;
    for (uint32_t c = threadIdx.x; c < gridDim.x; c += kFreeThreads) {
        const uint32_t x = __ldcg(P.counts + c);
        all += x;
        before += c < blockIdx.x ? x : 0u;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0) {
        sums[warp] = mine;
        before_sum[warp] = before;
        all_sum[warp] = all;
    }
    __syncthreads();
    uint32_t at = 0, total = 0;
    for (int w = 0; w < kFreeWarps; ++w) {
        at += before_sum[w] + (w < warp ? sums[w] : 0u);
        total += all_sum[w];
    }
    free_give(P, it, kept, head, at, total);
    if (blockIdx.x == 0 && threadIdx.x == 0) free_head(P, head0, head, total);
}

// ------------------------------------------------------------------ compact
// scratch: map[n] (1 where in use, then the new id), movers[n], holes[n], [L, moves]
struct CompactScratch {
    uint32_t *map, *movers, *holes, *counts;
};
__host__ __device__ inline CompactScratch compact_scratch(uint32_t* s, uint32_t n) {
    return {s, s + n, s + 2 * static_cast<size_t>(n), s + 3 * static_cast<size_t>(n)};
}

__device__ __forceinline__ uint32_t used_entries(const CompactPoolParams& P, uint32_t r, bool& ok) {
    const uint32_t n = blocks_of(__ldg(P.past + r), P.pool.block);
    ok = n <= P.bt_stride;
    return ok ? n : P.bt_stride;
}

// Which blocks are in use, how many (L), and the moves: the blocks in use from
// L on, in order, go to the free ids below L, in order.
__global__ void __launch_bounds__(kListThreads) slotkv_compact_plan_kernel(const CompactPoolParams P) {
    __shared__ ListScan scan;
    begin_dependent();
    const int lane = threadIdx.x & 31;
    const uint32_t n = P.pool.n_blocks;
    const CompactScratch S = compact_scratch(P.scratch, n);
    const uint32_t gt = blockIdx.x * kListThreads + threadIdx.x, nt = gridDim.x * kListThreads;
    for (uint32_t i = gt; i < n; i += nt) S.map[i] = 0;
    cluster_barrier();
    const EntryItems it = my_items(P.R, P.bt_stride);
    for (uint32_t i = it.begin; i < it.end; ++i) {
        const uint32_t r = i / it.per_row, e = (i % it.per_row) * 32 + lane;
        bool ok;
        const bool live = e < used_entries(P, r, ok);
        const uint32_t id = live ? __ldg(P.block_tables + static_cast<size_t>(r) * P.bt_stride + e) : 0u;
        const bool bad = !ok || (live && id >= n);
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(P.pool.status, kRange);
        if (live && id < n) S.map[id] = 1;
    }
    cluster_barrier();
    // ids in order over the warps, 32 at a time
    const uint32_t warps = gridDim.x * kListWarps, groups = (n + 31) / 32;
    const uint32_t per = (groups + warps - 1) / warps;
    const uint32_t w = blockIdx.x * kListWarps + (threadIdx.x >> 5);
    const uint64_t g0 = static_cast<uint64_t>(w) * per;
    const uint32_t b = static_cast<uint32_t>(g0 < groups ? g0 : groups);
    const uint32_t e = static_cast<uint32_t>(g0 + per < groups ? g0 + per : groups);
    uint32_t mine = 0;
    for (uint32_t g = b; g < e; ++g) {
        const uint32_t id = g * 32 + lane;
        mine += __popc(__ballot_sync(0xffffffffu, id < n && __ldcg(S.map + id) != 0u));
    }
    uint32_t L;
    const uint32_t first = cluster_exclusive(mine, scan, L);
    // blocks in use below L: found by the warp that holds id L
    uint32_t at = first;
    for (uint32_t g = b; g < e; ++g) {
        const uint32_t id = g * 32 + lane;
        const bool live = id < n && __ldcg(S.map + id) != 0u;
        const uint32_t m = __ballot_sync(0xffffffffu, live);
        const uint32_t before = at + __popc(m & ((1u << lane) - 1u));  // in use below id
        if (id == L) S.counts[1] = L - before;
        if (id < L && !live) S.holes[id - before] = id;
        at += __popc(m);
    }
    if (gt == 0) {
        S.counts[0] = L;
        if (L == n) S.counts[1] = 0;
    }
    cluster_barrier();
    const uint32_t below = L - __ldcg(S.counts + 1);
    at = first;
    for (uint32_t g = b; g < e; ++g) {
        const uint32_t id = g * 32 + lane;
        const bool live = id < n && __ldcg(S.map + id) != 0u;
        const uint32_t m = __ballot_sync(0xffffffffu, live);
        const uint32_t before = at + __popc(m & ((1u << lane) - 1u));
        if (id < n) {
            uint32_t to = id;
            if (live && id >= L) {
                to = __ldcg(S.holes + before - below);
                S.movers[before - below] = id;
            }
            S.map[id] = to;
            if (P.shares && id >= L && !live) P.shares[id] = 0;  // (the moves clear the others')
        }
        at += __popc(m);
    }
    // the ids from L on are the free list now
    const uint32_t left = n - L, F = left < P.n_free ? left : P.n_free;
    for (uint32_t i = gt; i < F; i += nt) P.free_blocks[P.n_free - F + i] = L + i;
    if (gt == 0) {
        *P.head = P.n_free - F;
        if (F < left) atomicOr(P.pool.status, kRange);
    }
}

// The same for a pool of up to 32 blocks per thread of one CTA: the blocks in use
// as bits in shared memory, a word per thread (the phases above are round trips
// to L2, these barriers).
// (Of the whole call, nothing to move: 5.1 us against the cluster's 8.5 at 32 blocks
// and entries, 6.9 / 10.6 at 4096, 13.1 / 12.6 at 16384, 21 / 15 at 32768.)
constexpr uint32_t kSmallPool = 32 * kListThreads, kSmallEntries = 16 * kListThreads;
__global__ void __launch_bounds__(kListThreads) slotkv_compact_small_kernel(const CompactPoolParams P) {
    __shared__ uint32_t bits[kListThreads], warp_sum[kListWarps], moves_sum;
    begin_dependent();
    const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5, n = P.pool.n_blocks;
    const CompactScratch S = compact_scratch(P.scratch, n);
    bits[t] = 0;
    if (t == 0) moves_sum = 0;
    __syncthreads();
    for (uint32_t i = t; i < P.R * P.bt_stride; i += kListThreads) {
        const uint32_t r = i / P.bt_stride;
        bool ok;
        if (i - r * P.bt_stride >= used_entries(P, r, ok)) continue;
        const uint32_t id = __ldg(P.block_tables + i);
        if (id < n) atomicOr(&bits[id / 32], 1u << (id % 32));
        if (!ok || id >= n) atomicOr(P.pool.status, kRange);
    }
    __syncthreads();
    const uint32_t live = bits[t], mine = __popc(live);
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= static_cast<uint32_t>(o)) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    const uint32_t w = warp_sum[lane];  // (kListWarps = 32)
    const uint32_t first = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u) + incl - mine;
    const uint32_t L = __reduce_add_sync(0xffffffffu, w);  // blocks in use
    // this word's ids below L, from L on, and below n
    auto under = [&](uint32_t end) {
        return end <= 32 * t ? 0u : end - 32 * t >= 32 ? 0xffffffffu : (1u << (end - 32 * t)) - 1u;
    };
    const uint32_t low = under(L), all = under(n), holes = ~live & low, movers = live & ~low;
    // a hole's place is the number of holes before it, a mover's that of the movers: of the
    // ids below its word, 32 t - first are free and first in use
    for (uint32_t m = holes; m; m &= m - 1) {
        const uint32_t b = __ffs(m) - 1;
        S.holes[32 * t - first + __popc(~live & ((1u << b) - 1u))] = 32 * t + b;
    }
    if (movers) atomicAdd(&moves_sum, __popc(movers));
    __syncthreads();  // (the holes too)
    const uint32_t moves = moves_sum, below = L - moves;
    for (uint32_t m = movers; m; m &= m - 1) {
        const uint32_t b = __ffs(m) - 1, k = first + __popc(live & ((1u << b) - 1u)) - below, id = 32 * t + b;
        S.movers[k] = id;
        S.map[id] = __ldcg(S.holes + k);
    }
    if (P.shares)
        for (uint32_t m = ~live & ~low & all; m; m &= m - 1) P.shares[32 * t + __ffs(m) - 1] = 0;
    const uint32_t left = n - L, F = left < P.n_free ? left : P.n_free;
    for (uint32_t i = t; i < F; i += kListThreads) P.free_blocks[P.n_free - F + i] = L + i;
    if (t == 0) {
        S.counts[0] = L;
        S.counts[1] = moves;
        *P.head = P.n_free - F;
        if (F < left) atomicOr(P.pool.status, kRange);
    }
}

// The moves, share counts and tables, over the whole GPU: CTAs take (block,
// part) pairs in turn, then table entries.  Bound by HBM: 796 MB read and written in
// 150 us with the plan and the tables (5.3 TB/s).
__global__ void __launch_bounds__(kCopyThreads) slotkv_compact_move_kernel(const CompactPoolParams P,
                                                                           uint32_t parts) {
    begin_dependent();
    const CompactScratch S = compact_scratch(P.scratch, P.pool.n_blocks);
    const uint32_t moves = __ldcg(S.counts + 1), L = __ldcg(S.counts);
    const uint64_t n4 = static_cast<uint64_t>(P.pool.block) * (P.pool.kv_dim / 4);
    const uint64_t work = static_cast<uint64_t>(moves) * parts;
    for (uint64_t i = blockIdx.x; i < work; i += gridDim.x) {
        const uint32_t k = static_cast<uint32_t>(i / parts), part = static_cast<uint32_t>(i % parts);
        const uint32_t src = __ldcg(S.movers + k), dst = __ldcg(S.holes + k);
        const uint32_t t = part * kCopyThreads + threadIdx.x, step = parts * kCopyThreads;
        copy_float4(reinterpret_cast<const float4*>(P.pool.K) + src * n4,
                    reinterpret_cast<float4*>(P.pool.K) + dst * n4, n4, t, step);
        copy_float4(reinterpret_cast<const float4*>(P.pool.V) + src * n4,
                    reinterpret_cast<float4*>(P.pool.V) + dst * n4, n4, t, step);
        if (P.shares && part == 0 && threadIdx.x == 0) {
            P.shares[dst] = P.shares[src];
            P.shares[src] = 0;
        }
    }
    const uint64_t gt = static_cast<uint64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
    const uint64_t nt = static_cast<uint64_t>(gridDim.x) * kCopyThreads;
    const uint64_t entries = static_cast<uint64_t>(P.R) * P.bt_stride;
    for (uint64_t i = gt; i < entries; i += nt) {
        bool ok;
        const uint32_t r = static_cast<uint32_t>(i / P.bt_stride);
        if (i % P.bt_stride >= used_entries(P, r, ok)) continue;
        const uint32_t id = P.block_tables[i];
        if (id >= L && id < P.pool.n_blocks) P.block_tables[i] = __ldcg(S.map + id);
    }
}

template <typename... A>
int launch_dependent(void (*kernel)(A...), dim3 grid, int threads, uint32_t cluster,
                     cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// CTAs of a list kernel over n items of 32: one where its warps have one each.
uint32_t list_ctas(uint64_t n) { return n <= kListWarps ? 1u : kListCtas; }
// Items up to which freeing is one cluster's work (one for each of its warps).  One
// launch against four: 5.8 us against 8.5 at 8 items, 9.0 / 9.3 at 64, 9.7 / 9.8 at
// 256, 13.5 / 10.1 at 512, 73 / 17 at 4096.
constexpr uint64_t kListItems = kListWarps * kListCtas;
// Forks up to which every CTA reads all lengths before its own (forks of two full
// blocks: 16.7 us against 16.9 with the count kernel at 2048, 20.7 / 17.9 at 2500, 40 / 28
// at 4096, 5355 / 354 at 65536), and the forks of a run beyond (with 2048 as one run
// 34 us at 4096, 433 at 65536).
constexpr uint32_t kForkOne = 2048;

}  // namespace

int launch_keep_path(const KeepPathParams& p, cudaStream_t stream) {
    const uint32_t cols = 2 * (p.pool.kv_dim / 4);
    const dim3 grid(p.R, (cols + kCopyThreads - 1) / kCopyThreads);
    return launch_dependent(slotkv_keep_path_kernel, grid, kCopyThreads, 0, stream, p);
}

int launch_fork_tables(const ForkTablesParams& p, uint32_t sms, cudaStream_t stream) {
    // enough parts for few forks to fill the GPU, none smaller than one batch of every thread
    const uint64_t most = (static_cast<uint64_t>(p.pool.block) * (p.pool.kv_dim / 4) + kBatch * kCopyThreads - 1) /
                          (kBatch * kCopyThreads);
    const uint32_t forks = p.n_fork ? p.n_fork : 1u;
    uint32_t parts = (4 * sms + forks - 1) / forks;
    parts = parts < most ? parts : static_cast<uint32_t>(most);
    parts = parts < 64u ? parts : 64u;
    const dim3 grid(forks, parts ? parts : 1u);
    if (forks <= kForkOne)
        return launch_dependent(slotkv_fork_tables_kernel<false>, grid, kCopyThreads, 0, stream, p);
    const int rc = launch_dependent(slotkv_fork_count_kernel, dim3((forks + kForkRun - 1) / kForkRun), kCopyThreads,
                                    0, stream, p);
    if (rc != 0) return rc;
    return launch_dependent(slotkv_fork_tables_kernel<true>, grid, kCopyThreads, 0, stream, p);
}

int launch_free_tables(const FreeTablesParams& p, uint32_t sms, cudaStream_t stream) {
    const uint64_t items = static_cast<uint64_t>(p.R) * ((p.bt_stride + 31) / 32);
    if (items <= kListItems) {
        const uint32_t ctas = list_ctas(items);
        return launch_dependent(slotkv_free_tables_kernel, dim3(ctas), kListThreads, ctas, stream, p);
    }
    const uint64_t want = (items + kFreeWarps - 1) / kFreeWarps, most = sms < kFreeCtas / 4 ? 4 * sms : kFreeCtas;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    int rc = 0;
    if (p.shares) {
        rc = launch_dependent(slotkv_free_take_kernel, grid, kFreeThreads, 0, stream, p);
        if (rc == 0) rc = launch_dependent(slotkv_free_sign_kernel, grid, kFreeThreads, 0, stream, p);
    }
    if (rc == 0) rc = launch_dependent(slotkv_free_count_kernel, grid, kFreeThreads, 0, stream, p);
    if (rc == 0) rc = launch_dependent(slotkv_free_give_kernel, grid, kFreeThreads, 0, stream, p);
    return rc;
}

int launch_compact_pool(const CompactPoolParams& p, uint32_t sms, cudaStream_t stream) {
    const uint64_t items = static_cast<uint64_t>(p.R) * ((p.bt_stride + 31) / 32);
    const uint64_t groups = (static_cast<uint64_t>(p.pool.n_blocks) + 31) / 32;
    int rc;
    if (p.pool.n_blocks <= kSmallPool && static_cast<uint64_t>(p.R) * p.bt_stride <= kSmallEntries) {
        rc = launch_dependent(slotkv_compact_small_kernel, dim3(1), kListThreads, 0, stream, p);
    } else {
        const uint32_t ctas = list_ctas(items > groups ? items : groups);
        rc = launch_dependent(slotkv_compact_plan_kernel, dim3(ctas), kListThreads, ctas, stream, p);
    }
    if (rc != 0) return rc;
    const uint64_t most = (static_cast<uint64_t>(p.pool.block) * (p.pool.kv_dim / 4) + kBatch * kCopyThreads - 1) /
                          (kBatch * kCopyThreads);
    const uint32_t parts = most < 8u ? static_cast<uint32_t>(most) : 8u;
    return launch_dependent(slotkv_compact_move_kernel, dim3(4 * sms), kCopyThreads, 0, stream, p, parts);
}

}  // namespace slotkv
