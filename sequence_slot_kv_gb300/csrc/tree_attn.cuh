// tree_attn.cuh -- attention of trees of drafted tokens over slots or a paged
// pool (tree_batch_attn, tree_batch_attn_paged).
//
// Request r holds past keys and brings n nodes; node i's key goes to place
// past + i of its slot, its position is past + depth(i), and it attends the
// past keys, its ancestors and itself:
//   out_i = sum_j e^(s_ij) V_j / (sum_j e^(s_ij) + e^sink),  s_ij the scaled
//   score after the call's rule (score_rule.cuh),
// over j < past and the nodes j whose bit is set in i's set of ancestors.
#pragma once

#include "decode_attn.cuh"
#include "tc_ops.cuh"
#include "tree_attn.h"

namespace slotkv {

// Place p of request r in the [rows][kv_dim] view (p in range, its block in the pool).
__device__ __forceinline__ uint32_t tree_row(const TreeParams& P, uint32_t r, uint32_t p) {
    if (P.block_tables)
        return __ldg(P.block_tables + static_cast<size_t>(r) * P.bt_stride + p / P.slot_ctx) * P.slot_ctx +
               p % P.slot_ctx;
    return __ldg(P.slots + r) * P.slot_ctx + p;
}

// The same for any place and any table: what is not in the pool is read from
// its first block instead (and belongs to a request that prep has refused).
__device__ __forceinline__ uint32_t tree_place(const TreeParams& P, uint32_t r, uint32_t p) {
    const uint32_t b = P.block_tables
                           ? __ldg(P.block_tables + static_cast<size_t>(r) * P.bt_stride + p / P.slot_ctx)
                           : __ldg(P.slots + r);
    return (b < P.n_slots ? b : 0u) * P.slot_ctx + (P.block_tables ? p % P.slot_ctx : p);
}

// ------------------------------------------------------------------ prep
// CTA (request, part), behind a column of CTAs whose first ones plan the attention
// kernel's work (tree_plan_ctas).  Every part checks the request and finds its nodes' depths
// by pointer doubling over the tree in shared memory (a round adds to a node's
// depth that of the node it points at and doubles the distance, so a chain of
// 256 takes 8 rounds).  Part 0 does the same with the sets of ancestors and
// writes, for every node, the set of the nodes that attend it.  The other parts
// form the request's vectors, one warp per (node, P.prep_heads query heads or half
// as many kv heads): q' = RoPE(RMSnorm(q) w) scale log2(e) into the
// workspace, k' and v into the node's cache row, with the decode kernel's
// vector routines (so the same bits as a decode step's at that position).  A
// call is bound by its dependent loads here; a warp's first rows are on their
// way while the tree is looked at.  A warp's heads come one after the other (0.4 us
// each, 1.6 at head dim 256), so it has as few as keep the grid at kPrepCtas CTAs an SM:
// 14 nodes of 8 heads 21.0 -> 19.4 us against 8 heads a warp, 27 nodes of 8 heads of
// 256 137 -> 132 (whole calls); calls too large for that keep 8, whose angles, table
// and tree are looked at once for all of them (620 nodes of 32 heads: 14 us, cold).
constexpr int kPrepHeads = 8, kPrepCtas = 4, kPrepThreads = 128, kPrepWarps = kPrepThreads / 32;

__device__ __forceinline__ void tree_cp_async16(void* smem_dst, const void* gmem_src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem_dst)), "l"(gmem_src)
                 : "memory");
}

// A request's first node, nodes, and whether it is in range (its parents apart).
struct TreeReq {
    uint32_t s0, n, past;
    bool ok;
};
__device__ __forceinline__ TreeReq tree_request(const TreeParams& P, uint32_t r) {
    TreeReq q;
    const uint32_t s1 = __ldg(P.starts + r + 1);
    q.s0 = __ldg(P.starts + r);
    q.past = __ldg(P.past + r);
    q.n = s1 - q.s0;
    uint64_t cap = P.block_tables ? static_cast<uint64_t>(P.bt_stride) * P.slot_ctx : P.slot_ctx;
    cap = cap < kTreePlaces ? cap : kTreePlaces;
    q.ok = q.s0 <= s1 && s1 <= P.n_tok && q.n <= kTreeNodes && static_cast<uint64_t>(q.past) + q.n <= cap;
    if (!P.block_tables) q.ok = q.ok && __ldg(P.slots + r) < P.n_slots;
    return q;
}

// ------------------------------------------------------------------ units
// What a role reads of a unit (or the part of it that the CTA has), in words of
// shared memory.  Tiles go from the last keys to the first: tile t of the part
// begins at place d[kPlace] - 128 t.
enum TreeWord { kReq, kRow, kNodes, kPast, kKvHead, kRow0, kRows, kPlace, kTiles, kStart, kWhole, kMore };

// The sets of 1 << k blocks of a request of nb, and the first block of the first.
constexpr int kSetSizes = 4;
__device__ __forceinline__ uint32_t tree_sets(uint32_t nb, int k) {
    return k == kSetSizes - 1 ? nb >> k : nb >> k & 1u;
}
__device__ __forceinline__ uint32_t tree_set_block(uint32_t nb, int k) {
    return k == kSetSizes - 1 ? 0u : nb & ~((2u << k) - 1u);
}
// A request's shape: row blocks, first tile, tiles; 0 blocks: nothing to do.
struct TreeShape {
    TreeReq q;
    uint32_t nb, tile0, tl;
    // tiles of its sets of 1 << k blocks
    __device__ uint64_t tiles(uint32_t n_kv_head, int k) const {
        return static_cast<uint64_t>(tree_sets(nb, k)) * tl * n_kv_head;
    }
};
template <int RB>
__device__ __forceinline__ TreeShape tree_shape(const TreeParams& P, uint32_t r) {
    TreeShape x;
    x.q = tree_request(P, r);
    x.nb = x.tile0 = x.tl = 0;
    if (!x.q.ok || x.q.n == 0) return x;
    const uint32_t last = x.q.past + x.q.n - 1, lo = rule_first(P.rule, r, x.q.past);
    x.nb = (x.q.n * (P.n_head / P.n_kv_head) + RB - 1) / RB;
    x.tile0 = (lo < last ? lo : last) / 128;
    x.tl = last / 128 - x.tile0 + 1;
    return x;
}

// The tiles of the sets of each size (one row block's), the groups of CTAs that
// share them, and the first CTA of the groups.
struct TreePlan {
    uint64_t total[kSetSizes];
    uint32_t groups[kSetSizes], first[kSetSizes];
};
__device__ __forceinline__ uint64_t divide(uint64_t a, uint64_t b) {  // (of 32 bits where they do)
    return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}
// As many groups as fit, so that the longest range is as short as may be.
__device__ __forceinline__ void tree_plan(TreePlan& p, uint32_t ctas) {
    uint64_t work = 0;
#pragma unroll
    for (int k = 0; k < kSetSizes; ++k) work += p.total[k] << k;
    int left = static_cast<int>(ctas);
#pragma unroll
    for (int k = 0; k < kSetSizes; ++k) {
        uint64_t g = p.total[k] ? divide(p.total[k] * ctas, work) : 0u;
        g = g < p.total[k] ? g : p.total[k];
        p.groups[k] = p.total[k] ? (g ? static_cast<uint32_t>(g) : 1u) : 0u;
        left -= static_cast<int>(p.groups[k] << k);
    }
    for (;;) {
        // the size with the longest ranges gets another group, or, where the groups of at
        // least one are too many, the one with the shortest loses one
        int best = -1;
#pragma unroll
        for (int k = 0; k < kSetSizes; ++k) {
            const bool can = left >= 0 ? (1 << k) <= left && p.groups[k] && p.groups[k] < p.total[k] : p.groups[k] > 1;
            if (!can) continue;
            if (best >= 0) {
                uint64_t a = 0, b = 0;  // total[k] / groups[k] against the best one's
#pragma unroll
                for (int x = 0; x < kSetSizes; ++x)
                    if (x == best) a = p.total[k] * p.groups[x], b = p.total[x] * p.groups[k];
                if (left >= 0 ? a <= b : a >= b) continue;
            }
            best = k;
        }
        if (best < 0) break;
#pragma unroll
        for (int k = 0; k < kSetSizes; ++k)
            if (k == best) p.groups[k] += left >= 0 ? 1u : -1u;
        left -= left >= 0 ? 1 << best : -(1 << best);
    }
    uint32_t at = 0;
#pragma unroll
    for (int k = 0; k < kSetSizes; ++k) {
        p.first[k] = at;
        at += p.groups[k] << k;
    }
}
// Every group has each tiles, the first over groups one more; the group of tile x.
__device__ __forceinline__ uint32_t tree_owner(uint64_t each, uint32_t over, uint64_t x) {
    const uint64_t cut = over * (each + 1);
    return static_cast<uint32_t>(x < cut ? divide(x, each + 1) : over + divide(x - cut, each));
}

// A CTA's parts of units, in order.
template <int RB>
struct TreeWalk {
    int k;               // the sets' size, 1 << k, and the block of a set that is this CTA's
    uint32_t member;
    uint32_t r;
    uint64_t off, left;  // tiles into request r, tiles left
    TreeShape x;
    bool known;
    __device__ bool next(const TreeParams& P, uint32_t (&d)[12]) {
        if (left == 0) return false;
        for (;;) {
            if (!known) {
                if (r >= P.n_req) return false;
                x = tree_shape<RB>(P, r);
                known = true;
            }
            const uint64_t n = x.tiles(P.n_kv_head, k);
            if (off < n) break;
            off -= n;
            ++r;
            known = false;
        }
        const uint32_t unit = static_cast<uint32_t>(divide(off, x.tl)), sets = tree_sets(x.nb, k);
        const uint32_t t0 = static_cast<uint32_t>(off - static_cast<uint64_t>(unit) * x.tl);
        const uint32_t n = left < x.tl - t0 ? static_cast<uint32_t>(left) : x.tl - t0;
        const uint32_t row0 = (tree_set_block(x.nb, k) + (unit % sets << k) + member) * RB;
        const uint32_t all = x.q.n * (P.n_head / P.n_kv_head) - row0;
        d[kReq] = r;
        d[kRow] = x.q.s0;
        d[kNodes] = x.q.n;
        d[kPast] = x.q.past;
        d[kKvHead] = unit / sets;
        d[kRow0] = row0;
        d[kRows] = all < RB ? all : RB;
        d[kPlace] = (x.tile0 + x.tl - 1 - t0) * 128;
        d[kTiles] = n;
        d[kStart] = t0 == 0 ? 1u : 0u;
        d[kWhole] = n == x.tl ? 1u : 0u;
        d[kMore] = 1u;
        off += n;
        left -= n;
        return true;
    }
};

// Where every CTA of the attention kernel begins, by the first CTAs of the prep kernel,
// a thread per CTA: the totals of the sizes, the plan, then the requests' first tiles,
// 128 requests at a time, among which a CTA finds its own.  (When each CTA of the
// attention kernel did this for itself, its first unit was known 3 to 9 us after prep's
// end: the code runs once, from cold instruction caches.)
template <int RB>
__device__ void tree_plan_ctas(const TreeParams& P) {
    constexpr uint32_t NT = kPrepThreads, NW = NT / 32;
    static_assert(NT == 128, "a power of two that the search halves");
    __shared__ uint64_t begin[kSetSizes][NT];  // the requests' first tiles
    __shared__ uint64_t sums[kSetSizes][NW], totals[kSetSizes], each[kSetSizes];
    __shared__ uint32_t over[kSetSizes], groups[kSetSizes], first_cta[kSetSizes];
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const TreeShape first = tid < P.n_req ? tree_shape<RB>(P, tid) : TreeShape{};
    // (loops over the sizes stay loops where they can: this code runs once, from cold
    // instruction caches)
#pragma unroll 1
    for (int k = 0; k < kSetSizes; ++k) {
        uint64_t all = first.tiles(P.n_kv_head, k);
        for (uint32_t r = tid + NT; r < P.n_req; r += NT) all += tree_shape<RB>(P, r).tiles(P.n_kv_head, k);
        if (__any_sync(0xffffffffu, all != 0))
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        if (lane == 0) sums[k][warp] = all;
    }
    __syncthreads();
    if (warp == 0) {
        TreePlan plan;
#pragma unroll
        for (int k = 0; k < kSetSizes; ++k) {
            plan.total[k] = 0;
#pragma unroll
            for (uint32_t w = 0; w < NW; ++w) plan.total[k] += sums[k][w];
        }
        tree_plan(plan, P.ctas);
        uint64_t t = 0;
        uint32_t g = 0, f = 0;  // this lane's size
#pragma unroll
        for (uint32_t k = 0; k < kSetSizes; ++k)
            if (lane == k) t = plan.total[k], g = plan.groups[k], f = plan.first[k];
        const uint64_t q = divide(t, g ? g : 1u);
        if (lane < kSetSizes) {
            totals[lane] = t;
            each[lane] = q;
            over[lane] = static_cast<uint32_t>(t - q * g);
            groups[lane] = g;
            first_cta[lane] = f;
        }
    }
    __syncthreads();
    for (uint32_t c0 = blockIdx.y * NT; c0 < P.ctas; c0 += gridDim.y * NT) {
        const uint32_t cta = c0 + tid;
        TreeWalk<RB> walk;
        walk.known = false;
        walk.k = 0;
        walk.r = walk.member = 0;
        walk.off = walk.left = 0;
        uint64_t u0 = 0;
#pragma unroll 1
        for (int k = 0; k < kSetSizes; ++k) {
            const uint32_t c = cta - first_cta[k], group = c >> k;
            if (cta >= P.ctas || cta < first_cta[k] || group >= groups[k]) continue;
            walk.k = k;
            walk.member = c & ((1u << k) - 1u);
            u0 = group * each[k] + min(group, over[k]);
            walk.left = each[k] + (group < over[k] ? 1u : 0u);
        }
        const uint64_t u1 = u0 + walk.left;
        bool found = walk.left == 0;
        uint64_t at = 0;  // of this CTA's size, up to this 128 requests
        for (uint32_t r0 = 0; r0 < P.n_req; r0 += NT) {
            const uint32_t r = r0 + tid;
            const TreeShape x = !r0 ? first : r < P.n_req ? tree_shape<RB>(P, r) : TreeShape{};
            __syncthreads();  // (the last ones have been searched)
#pragma unroll 1
            for (int k = 0; k < kSetSizes; ++k) {
                if (totals[k] == 0) continue;
                const uint64_t n = x.tiles(P.n_kv_head, k);
                uint64_t incl = n;
#pragma unroll
                for (uint32_t o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                begin[k][tid] = incl - n;  // in the warp
                if (lane == 31) sums[k][warp] = incl;
            }
            __syncthreads();
            // the warp that this CTA's first tile is in, and the request there
            uint64_t before = at;
            uint32_t w = 0;
            for (; w < NW && !found; ++w) {
                if (u0 < before + sums[walk.k][w]) break;
                before += sums[walk.k][w];
            }
            if (!found && w < NW) {
                uint32_t i = 32 * w;  // the last one that begins there or before
#pragma unroll
                for (uint32_t o = 16; o > 0; o >>= 1)
                    if (before + begin[walk.k][i + o] <= u0) i += o;
                walk.r = r0 + i;
                walk.off = u0 - before - begin[walk.k][i];
                found = true;
            }
            at = before;
            if (__syncthreads_and(found)) break;
        }
        if (cta >= P.ctas) continue;
        uint32_t d[12] = {};
        uint32_t* to = P.plan + kTreePlan * static_cast<size_t>(cta);
        d[kMore] = walk.next(P, d) ? 1u : 0u;
#pragma unroll
        for (int i = 0; i < 12; ++i) to[i] = d[i];
        to[kPlanUnitTiles] = d[kMore] ? walk.x.tl : 0u;
        to[kPlanSize] = walk.k;
        to[kPlanMember] = walk.member;
        to[kPlanReq] = walk.r;
        to[kPlanOver] = over[walk.k];
        const uint64_t wide[4] = {walk.off, walk.left, u1, each[walk.k]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            to[kPlanOff + 2 * i] = static_cast<uint32_t>(wide[i]);
            to[kPlanOff + 2 * i + 1] = static_cast<uint32_t>(wide[i] >> 32);
        }
    }
}

// ------------------------------------------------------------------ prep kernel
template <int HD>
__global__ void __launch_bounds__(kPrepThreads) slotkv_tree_prep_kernel(const TreeParams P) {
    extern __shared__ __align__(16) uint8_t prep_smem[];
    __shared__ uint32_t set[kTreeNodes][kTreeWords];
    __shared__ uint32_t jump[kTreeNodes], depth[kTreeNodes];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0) {
        if (blockIdx.y * kPrepThreads < P.ctas) tree_plan_ctas<static_cast<int>(tree_rows(HD))>(P);
        return;
    }
    const uint32_t r = blockIdx.x - 1;
    const bool sets = blockIdx.y == 0;
    const TreeReq q = tree_request(P, r);
    if (q.n == 0) return;
    // this warp's rows of item it, on their way
    const uint32_t qh = P.prep_heads, kvh = (qh + 1) / 2;
    const uint32_t qg = (P.n_head + qh - 1) / qh;
    const uint32_t groups = qg + (P.n_kv_head + kvh - 1) / kvh;
    float* rows = reinterpret_cast<float*>(prep_smem) + warp * 2 * kvh * HD;
    float* vrows = rows + kvh * HD;
    struct Item {
        uint32_t node, x0, nx;
        bool is_q;
    };
    auto item = [&](uint32_t it) {
        Item m;
        const uint32_t grp = it % groups;
        m.node = it / groups;
        m.is_q = grp < qg;
        m.x0 = m.is_q ? grp * qh : (grp - qg) * kvh;
        const uint32_t left = (m.is_q ? P.n_head : P.n_kv_head) - m.x0, most = m.is_q ? qh : kvh;
        m.nx = left < most ? left : most;
        return m;
    };
    auto load = [&](const Item& m) {
        const size_t tok = q.s0 + m.node;
        const float* src = m.is_q ? P.q + (tok * P.n_head + m.x0) * HD : P.k_new + (tok * P.n_kv_head + m.x0) * HD;
        const float* vsrc = P.v_new + (tok * P.n_kv_head + m.x0) * HD;
        for (uint32_t c = lane; c < m.nx * (HD / 4); c += 32) {
            tree_cp_async16(rows + 4 * c, src + 4 * c);
            if (!m.is_q) tree_cp_async16(vrows + 4 * c, vsrc + 4 * c);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const uint32_t step = (gridDim.y - 1) * kPrepWarps;
    uint32_t it = sets || !q.ok ? 0xFFFFFFFFu : (blockIdx.y - 1) * kPrepWarps + warp;
    const uint32_t items = q.ok ? q.n * groups : 0u;
    if (it < items) load(item(it));
    // the request's table and tree
    bool ok = q.ok;
    if (ok && P.block_tables) {
        const uint32_t used = (q.past + q.n - 1) / P.slot_ctx + 1;
        for (uint32_t e = tid; e < used; e += kPrepThreads)
            ok = ok && __ldg(P.block_tables + static_cast<size_t>(r) * P.bt_stride + e) < P.n_slots;
    }
    if (q.ok) {
        for (uint32_t i = tid; i < q.n; i += kPrepThreads) {
            const uint32_t p = __ldg(P.parents + q.s0 + i);
            const bool root = p == kTreeSkip;
            ok = ok && (root || p < i);
            jump[i] = root || p >= i ? kTreeSkip : p;
            depth[i] = root ? 0u : 1u;
            if (sets)
#pragma unroll
                for (uint32_t w = 0; w < kTreeWords; ++w) set[i][w] = i / 32 == w ? 1u << (i % 32) : 0u;
        }
    }
    ok = __syncthreads_and(ok) != 0;
    if (!ok) {
        if (sets) {
            if (tid == 0) atomicOr(P.status, kDevRange);
            if (q.s0 + q.n <= P.n_tok && q.n <= P.n_tok)  // (no more than the rows there are)
                for (uint32_t i = tid; i < q.n; i += kPrepThreads) P.req_of[q.s0 + i] = kTreeSkip;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        return;
    }
    constexpr int PER = kTreeNodes / kPrepThreads;
    const uint32_t words = sets ? (q.n + 31) / 32 : 0u;
    for (uint32_t far = 1; far < q.n; far *= 2) {
        uint32_t j[PER], d[PER] = {}, to[PER] = {}, s[PER][kTreeWords] = {};
        bool any = false;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const uint32_t i = tid + k * kPrepThreads;
            j[k] = i < q.n ? jump[i] : kTreeSkip;
            if (j[k] == kTreeSkip) continue;
            any = true;
            d[k] = depth[j[k]];
            to[k] = jump[j[k]];
#pragma unroll
            for (uint32_t w = 0; w < kTreeWords; ++w)
                if (w < words) s[k][w] = set[j[k]][w];
        }
        if (!__syncthreads_or(any)) break;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (j[k] == kTreeSkip) continue;
            const uint32_t i = tid + k * kPrepThreads;
            depth[i] += d[k];
            jump[i] = to[k];
#pragma unroll
            for (uint32_t w = 0; w < kTreeWords; ++w)
                if (w < words) set[i][w] |= s[k][w];
        }
        __syncthreads();
    }
    if (sets) {
        for (uint32_t i = tid; i < q.n; i += kPrepThreads) {
            P.req_of[q.s0 + i] = r;
            P.depth[q.s0 + i] = depth[i];
        }
        // transposed, 32 x 32 nodes at a time: a lane has a node's ancestors, a vote each
        // ancestor's lane
        for (uint32_t b = warp; b < words * words; b += kPrepWarps) {
            const uint32_t wi = b / words, wj = b % words, i = 32 * wi + lane;
            const uint32_t v = i < q.n ? set[i][wj] : 0u;
            uint32_t mine = 0;
#pragma unroll
            for (uint32_t k = 0; k < 32; ++k) {
                const uint32_t y = __ballot_sync(0xffffffffu, v >> k & 1u);
                mine = lane == k ? y : mine;
            }
            if (32 * wj + lane < q.n) P.below[static_cast<size_t>(q.s0 + 32 * wj + lane) * kTreeWords + wi] = mine;
        }
        return;
    }
    const float w1 = (P.flags & kOptNormPlusOne) ? 1.0f : 0.0f;
    for (; it < items; it += step) {
        const Item m = item(it);
        float cs[HD / 64], sn[HD / 64];
        warp_rope_angles<HD>(q.past + depth[m.node], P.inv_freq, cs, sn, lane);
        const size_t at = m.is_q ? (static_cast<size_t>(q.s0 + m.node) * P.n_head + m.x0) * HD
                                 : (static_cast<size_t>(tree_row(P, r, q.past + m.node)) * P.n_kv_head + m.x0) * HD;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        for (uint32_t x = 0; x < m.nx; ++x) {
            if (m.is_q) {
                warp_norm_rope<HD>(rows + x * HD, P.q_rot + at + x * HD, P.q_norm_w, w1, P.scale_log2, P.eps, cs, sn,
                                   lane);
                continue;
            }
            warp_norm_rope<HD>(rows + x * HD, P.K + at + x * HD, P.k_norm_w, w1, 1.0f, P.eps, cs, sn, lane);
            if (P.flags & kOptVNorm) {
                warp_rms_norm_plain<HD>(vrows + x * HD, P.V + at + x * HD, P.eps, lane);
            } else {
#pragma unroll
                for (int j = 0; j < HD / 32; ++j) P.V[at + x * HD + lane + 32 * j] = vrows[x * HD + lane + 32 * j];
            }
        }
        __syncwarp();
        if (it + step < items) load(item(it + step));
    }
}

// ------------------------------------------------------------------ attention
// Persistent, one CTA per SM, on the tensor cores.  A unit of work is one
// (request, kv head, block of RB query rows), a row being a (node, query head of
// the kv head) pair; its keys come in tiles of 128.  Few rows meet many keys
// here, so the keys are the MMA's M: S^T[128 keys][rows] = K Q^T and
// O^T[hd][rows] = V^T P^T, N = the block's rows rounded up to 16.  (With the rows
// as M, as the prefill has them, a block of 40 rows would cost as much as one of
// 128.)
//
// f32 accuracy from TF32 products: a = a_hi + a_lo, a.b ~ a_hi.b_hi + a_hi.b_lo +
// a_lo.b_hi.  The hi and lo parts of Q and P stand one after the other in shared
// memory, so that one MMA with twice the N makes a_hi.b_hi and a_hi.b_lo; the
// sums of the products with a low part have columns of their own, where nothing
// large cuts their bits off, and join the others in registers.  A TF32 operand's
// f32 bits are read with the low 13 mantissa bits ignored, so a value is its own
// high part.
//   All of these cuts are toward zero, so they do not average out: left alone the
// outputs were 0.6, 0.85 and 1.2e-6 too small at head dims 64, 128 and 256, most of
// their error.  For O what is put back goes by what was cut, so that a row gets
// its V to the bit where nothing is (one key, or keys of one weight, and V of 11
// bits).  P's high part is cut from P (1 + 0.36 2^-10): where half of its last place
// is on average, so that P's low part has both signs, and neither the bits cut off
// that nor its product with V's low part, which is left out, adds up.  (A P of 11
// bits stays: 0.36 2^-10 of it is below its last place.)  Of V's 13 low bits 11 are
// read: of 4094.6 units that is on average 0.875 too few (3/2 where bit 12 is the
// highest, 1/2 where 11 is), so the sums of products with a low part count 1 +
// 0.875 / 4094.6 times.
//   S: a step of a chain of n (eight products each) cuts its sum by half a
// unit in the last place, 0.36 2^-23 of it on average; a dominant key's score grows
// evenly, so it ends 0.18 (n + 1) 2^-23 too small, n = hd / 8, which joining the two
// sums multiplies back.  That is one factor for all scores, so it moves a weight
// by that part of its distance from the row's highest score; between a key whose
// product with q grows evenly and one that has it in the last channels, which
// loses nothing, what was cut from the first remains, with the factor or without.
//   Over 80 drawn cases the outputs' relative error (root mean square) is 0.8 to
// 5.5e-7, between 2.6e-7 too small and 0.8e-7 too large (left alone up to 1.4e-6; the
// plain f32 form's goes up to 1.4e-6).
//   The A operands come from tensor memory, where a warp's lanes are
// the operand's rows: K is written there by the thread that owns the key, V^T by
// the thread that owns the dim, which makes the transposition free (and K's
// piece of the ring free again as soon as it has been read; MMAs that take A
// from shared memory too leave everyone else little of its bandwidth).  At head
// dim 64 one A holds V^T's high part in lanes 0-63
// and its low part in lanes 64-127, and one MMA forms all four products.
//
// Roles (eight warpgroups; the converters' and the last one's registers go to
// the accumulators):
//   0-3   softmax: a thread per key of the tile, each warpgroup every fourth group
//         of 8 rows.  Q rows into shared memory at a unit's start; then per tile S
//         from tensor memory, the rule and the masks, P^T (hi, lo) into shared
//         memory, the rows' sums in registers.  The running maxima are raised
//         lazily (by 2^8), the 128 threads agreeing at a named barrier.  (Beside the
//         MMAs shared memory answers after 200 cycles and more, which more warps
//         hide.)
//   4     accumulators: a thread per dim.  Every tile's O^T starts anew in
//         tensor memory (its chain of sums is cut toward zero at each step) and
//         is added to registers with rounded adds.  At the end out, or the
//         unit's partial result.
//   5, 6  converters, a piece each by turns: K and V^T (hi, lo) into tensor memory.
//   7     producer (16 KB pieces of K, 128 keys x 32 dims, swizzled, and of V by TMA
//         into a ring), two MMA issuers, and a warp that goes through the CTA's
//         units from there on and tells the others.
// The pieces go K(0), K(1), V(0), K(2), V(1), ... through the ring and through four
// buffers of tensor memory: S(t + 1) is formed while the softmax of tile t runs.
// (With two buffers for K's pieces and two for V's a converting warpgroup waited for
// the MMAs after every piece: 32 requests of 64 nodes took 2.64 ms, now 2.22.)
// P is handed over by blocks of 32 keys (a warp of each softmax warpgroup
// writes one), so tile t + 1's first blocks are written while the MMAs read
// tile t's last ones. A unit's tiles go from its last keys to its first, so
// that a distance bias raises no maximum tile after tile.
//
// A request's row blocks all read the same keys, so they are given out in sets of
// 8, 4, 2 and 1 (the binary digits of their number): the CTAs of a group take
// the blocks of a set side by side, tile for tile, and the keys come from memory
// once for all of them.  The tiles of all sets of one size, in order, are cut into
// one equal range per group, the CTAs divided among the sizes by their work
// (tree_plan; the prep kernel finds where each CTA begins).  So a unit may lie
// in several CTAs; each leaves (m, l, O) then, and slotkv_tree_combine_kernel
// joins them in the groups' order.
//
// What bounds it.  24 requests of 4000 keys, 8 kv heads of 128: 8 rows a kv head in
// 144 us, 5.5 TB/s (HBM, at 81 % of what a copy has with all of the call's three
// kernels counted); 64 rows 163; 128 rows 276; 256 rows 517, 512 rows 1038: 3.2 us for a
// tile of 64 rows and 128 keys, 6200 cycles, of which the MMAs alone take 3450 (they
// are active 55 % of the kernel's time).  The rest is the converters, 81 % busy with
// latencies (shared memory that the MMAs, TMA, P and they share, tensor memory,
// barriers), in issue slots that are 64 % used; what waits on them fills the other
// roles' time.  256 rows read 837 MB from HBM, K and V once (3.2 GB without the sets above).
//   8 kv heads of 64: 8 rows 104 us, 64 rows 124, 256 rows 398, 512 rows 806: 2.5 us a
// tile of 64 rows, MMAs 40 %, converters 83 %, issue slots 69 %.  4 kv heads of 256: 8 rows
// 139 us (5.7 TB/s), 32 rows 147, 54 rows 194, 256 rows 707: 4.4 us a tile of 32 rows, twice
// the bytes of one of 128, each block's CTA converting all of them (54 rows: MMAs
// 36 %, issue slots 53 %).
//   Code size counts: the roles run different code side by side, and what does not fit the
// instruction caches is fetched again every tile (the producer's loop unrolled costs
// 5 to 15 %).  In the 64 registers of the launch 20 words of a thread are spilled at head
// dim 128, 13 at 64 and none at 256.
//
// Keys past the request's last are zeros in V; a masked key's P is -0.  A V value
// that is not finite is a 0 to the tensor core, and the accumulators add it to
// the rows that attend its key (P not -0), so it reaches no other row.
//
// Every wait is bounded.  Where one runs out, its CTA raises SLOTKV_DEV_TIMEOUT
// and sets a flag that ends all its other waits at once; the roles go through
// the rest of their loops without doing anything, so they meet at their barriers
// and at the end as ever.  Such a CTA writes nothing from there on (a role that
// gave up hands on what it has not formed, so the accumulators look at the flag,
// not at their own waits alone) and says so beside its unit to join; the
// combine kernel leaves the rows alone that such a CTA has a part of.
template <int HD>
struct TreeCfg {
    static constexpr int KT = 128;                      // keys per tile
    static constexpr int RB = tree_rows(HD);            // rows per block
    static constexpr int PIECE = 16384;                 // bytes of a piece of K or V
    static constexpr int KP = HD / 32;                  // K pieces of a tile
    static constexpr int VD = tree_v_dims(HD);          // dims of a V piece
    static constexpr int VK = tree_v_keys(HD);          // keys of a V piece
    static constexpr int DH = HD / VD;                  // V pieces side by side
    static constexpr int VP = KT / VK * DH;             // V pieces of a tile
    static constexpr bool FOLD = HD == 64;              // V^T hi and lo in one A operand
    static constexpr int QBYTES = 2 * RB * HD * 4, PBYTES = 2 * RB * KT * 4;
    static constexpr int OFF_P = QBYTES, OFF_RING = QBYTES + PBYTES;
    static constexpr int NSLOT = (224 * 1024 - OFF_RING) / PIECE;  // 8, 6, 8
    static constexpr int NB = 4;                        // buffers of pieces in tensor memory
    // tensor memory columns; a buffer: K's hi | lo, 32 dims each, or V^T's, 32 keys each (FOLD: 64 keys)
    static constexpr int C_S = 0, C_O = 2 * RB, C_B = C_O + DH * 2 * RB, BCOLS = 64;
    static_assert(C_B + NB * BCOLS <= 512, "tensor memory");
    static constexpr int TMEM_COLS = 512;
    // what a chain of S's high products loses on average, and V's low parts (see above)
    static constexpr float ULP = 1.1920929e-7f;
    static constexpr float UNCUT_S = 1.f + static_cast<int>(0.18 * (HD / 8 + 1) + 0.5) * ULP;
    static constexpr float UNCUT_V = 1.f + 0.875f / 4094.625f;
    // shared memory behind the ring: row data, scratch of the maxima, barriers, flags
    static constexpr int OFF_M = OFF_RING + NSLOT * PIECE;      // running maxima [2 units][RB]
    static constexpr int OFF_F = OFF_M + 2 * RB * 4;            // factors of a raise, of the end [RB]
    static constexpr int OFF_POS = OFF_F + RB * 4;              // rows' positions [RB]
    static constexpr int OFF_SLOPE = OFF_POS + RB * 4;          // rows' slopes [RB]
    static constexpr int OFF_NODE = OFF_SLOPE + RB * 4;         // rows' nodes, from the block's first (bytes) [RB]
    static constexpr int OFF_MAX = OFF_NODE + RB;          // a warp's maxima, its sums [4][RB]
    static constexpr int OFF_DESC = OFF_MAX + 4 * RB * 4;       // what the roles need to know of a unit [2]
    static constexpr int OFF_BAR = OFF_DESC + 2 * 12 * 4;
    // piece landed, slot empty [NSLOT]; K in a buffer, V^T in it, the buffer empty [NB] (each kind's
    // issuer has to see every phase of the barrier that it waits at); S full, empty; P full, empty [4];
    // tile done with; O full, empty; Q full; unit's end; drain [2]; unit known, done with [2]
    static constexpr int NBAR = 2 * NSLOT + 3 * NB + 21;
    static constexpr int OFF_MISC = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;
    static constexpr int SMEM = OFF_MISC + 64;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static constexpr int CW = RB / 4;                   // rows of a softmax warpgroup
    static_assert(OFF_BAR % 8 == 0 && NSLOT >= 6, "layout");
};
constexpr int kTreeWarps = 32, kTreeThreads = 32 * kTreeWarps;
// registers of a thread: at launch (and of the softmax), and of the others from there on
constexpr int kTreeRegs = 64, kRegAcc = 112, kRegConv = 48, kRegAux = 48;
static_assert(4 * kTreeRegs + kRegAcc + 2 * kRegConv + kRegAux == kTreeWarps / 4 * kTreeRegs,
              "register hand-over must add up to the launch's registers");

__device__ __forceinline__ bool bar_or(int id, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(p)), "r"(id)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void bar_128(int id) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ float tree_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 lds4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// A word of shared memory at addr + at.
__device__ __forceinline__ void sts(uint32_t addr, int at, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr + at), "f"(v) : "memory");
}
// Packed f32x2 forms (each element rounded as the scalar operation would be).
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    return __ffma2_rn(b, make_float2(-1.f, -1.f), a);
}
// a times uncut, and b.
__device__ __forceinline__ float2 join2(float2 a, float2 b, float uncut) {
    return __ffma2_rn(a, make_float2(uncut, uncut), b);
}
// x without its low 13 mantissa bits: what the tensor core reads of it.
__device__ __forceinline__ uint32_t tf32_part(float x) { return __float_as_uint(x) & 0xFFFFE000u; }
// The low parts of two values.
__device__ __forceinline__ float2 low2(float x, float y) {
    return sub2(make_float2(x, y), make_float2(__uint_as_float(tf32_part(x)), __uint_as_float(tf32_part(y))));
}
// What the tensor core reads as P's high parts (see above).
__device__ __forceinline__ float2 near2(float x, float y) {
    return __ffma2_rn(make_float2(x, y), make_float2(0.36f / 1024.f, 0.36f / 1024.f), make_float2(x, y));
}

template <int HD, bool SC>
__global__ void __launch_bounds__(kTreeThreads, 1)
    slotkv_tree_attn_kernel(const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const TreeParams P) {
    using C = TreeCfg<HD>;
    constexpr int RB = C::RB, NSLOT = C::NSLOT;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t sbase = smem_addr(smem);
    volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
    // misc: [0] abort, [1] tensor memory; tiles (plus 1): [4 + 4 (tile & 1) + block] the last with a
    // V value that is not finite in that block of 32 keys, [12 + softmax warpgroup] the last
    // with a raise
    const uint32_t bar0 = sbase + C::OFF_BAR;
    const uint32_t RF = bar0, RE = RF + 8 * NSLOT, KF = RE + 8 * NSLOT, VF = KF + 8 * C::NB, BE = VF + 8 * C::NB,
                   SF = BE + 8 * C::NB, SE = SF + 8, PF = SE + 8, PE = PF + 32, FX = PE + 32, OF = FX + 8,
                   OE = OF + 8, QF = OE + 8, UE = QF + 8, DRAIN = UE + 8, GF = DRAIN + 16, GE = GF + 16;
    if (tid == 0) {
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(RF + 8 * i, 1);
            mbar_init(RE + 8 * i, 4);
        }
        for (int i = 0; i < C::NB; ++i) {
            mbar_init(KF + 8 * i, 4);
            mbar_init(VF + 8 * i, 4);
            mbar_init(BE + 8 * i, 1);
        }
        mbar_init(SF, 1);
        mbar_init(SE, 16);
        for (int i = 0; i < 4; ++i) {
            mbar_init(PF + 8 * i, 4);
            mbar_init(PE + 8 * i, 1);
        }
        mbar_init(FX, 4);
        mbar_init(OF, 1);
        mbar_init(OE, 4);
        mbar_init(QF, 16);
        mbar_init(UE, 4);
        mbar_init(DRAIN, 1);
        mbar_init(DRAIN + 8, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(GF + 8 * i, 1);
            mbar_init(GE + 8 * i, 31);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < 16; ++i) misc[i] = 0;
    }
    if (warp == 29) {
        tc::tmem_alloc(sbase + C::OFF_MISC + 4, C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tb = __shfl_sync(0xffffffffu, misc[1], 0);

    // A bounded wait; once the CTA has given up every wait ends at once.  (As little
    // code as may be: it stands in many places.)
    auto wait = [&](uint32_t bar, uint32_t parity) {
        uint32_t start = 0;
#pragma unroll 1
        for (uint32_t it = 0; it < (1u << 26); ++it) {
            if (mbar_try_wait(bar, parity)) return true;
            if (misc[0]) return false;
            const uint32_t now = static_cast<uint32_t>(clock());
            start = it ? start : now;
            if (now - start > 1u << 31) break;
        }
        misc[0] = 1;
        return false;
    };
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    // unit k of the CTA: its words, once they are there; done with them
    auto words = [&](uint32_t k) {
        return reinterpret_cast<const volatile uint32_t*>(smem + C::OFF_DESC) + 12 * (k & 1);
    };
    auto known = [&](uint32_t k) { return warp_wait(GF + 8 * (k & 1), (k >> 1) & 1); };
    auto done = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(GE + 8 * (k & 1));
    };
    const uint32_t G = P.n_head / P.n_kv_head;

    if (warp < 16) {
        // ------------------------------------------------------------ softmax
        grid_dependency_wait();
        constexpr int CW = C::CW;
        const int sg = warp >> 2, key = tid & 127, wq = warp & 3;  // warpgroup, key of the tile, lane quarter
        const int bar_id = 1 + sg;
        // row of the block of this warpgroup's row c
        auto row_of = [&](int c) { return 32 * (c / 8) + 8 * sg + c % 8; };
        float* fs = reinterpret_cast<float*>(smem + C::OFF_F) + 8 * sg;
        float* tmax = reinterpret_cast<float*>(smem + C::OFF_MAX);
        uint32_t* posr = reinterpret_cast<uint32_t*>(smem + C::OFF_POS) + 8 * sg;
        float* sloper = reinterpret_cast<float*>(smem + C::OFF_SLOPE) + 8 * sg;
        uint8_t* noder = smem + C::OFF_NODE + 8 * sg;
        const uint32_t tlane = tb + (static_cast<uint32_t>(wq) << 21);
        bool ok = true;
        uint32_t gt = 0;  // tiles so far
        for (uint32_t u = 0;; ++u) {
            ok = known(u) && ok;
            const volatile uint32_t* d = words(u);
            // (the four warps go on, or leave, together)
            if (bar_or(bar_id, !ok || !d[kMore])) break;
            const uint32_t rows = d[kRows], Rp = (rows + 15) / 16 * 16;
            float* ms = reinterpret_cast<float*>(smem + C::OFF_M) + (u & 1) * RB + 8 * sg;
            // Q rows, split with rounded high parts: [32-dim blocks][hi rows | lo rows][128 B].
            // (The last S has been read, so no MMA reads the last unit's Q.)
            constexpr int F4 = HD / 4, QN = RB * F4 / 512;  // float4s of a row, of a thread
            float4 qv[QN];
#pragma unroll
            for (int k = 0; k < QN; ++k) {
                const uint32_t row = (tid + 512 * k) / F4, at = d[kRow0] + row;
                qv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row < rows)
                    qv[k] = *reinterpret_cast<const float4*>(
                        P.q_rot + (static_cast<size_t>(d[kRow] + at / G) * P.n_head + d[kKvHead] * G + at % G) * HD +
                        4 * (tid % F4));
            }
            if (key < CW) {
                const uint32_t row = d[kRow0] + min(static_cast<uint32_t>(row_of(key)), rows - 1);
                const uint32_t pos = d[kPast] + P.depth[d[kRow] + row / G];
                const int at = row_of(key) - 8 * sg;
                ms[at] = -1e30f;
                posr[at] = pos;
                noder[at] = static_cast<uint8_t>(row / G - d[kRow0] / G);
                if (SC) sloper[at] = P.rule.slopes ? __ldg(P.rule.slopes + d[kKvHead] * G + row % G) * kRuleLog2e : 0.f;
            }
#pragma unroll
            for (int k = 0; k < QN; ++k) {
                const uint32_t row = (tid + 512 * k) / F4, c = tid % F4;
                if (row >= Rp) continue;
                uint4 hi, lo;
                auto split = [](float v, uint32_t& a, uint32_t& b) {
                    a = (__float_as_uint(v) + 0x1000u) & 0xFFFFE000u;
                    b = __float_as_uint(v - __uint_as_float(a));
                };
                split(qv[k].x, hi.x, lo.x);
                split(qv[k].y, hi.y, lo.y);
                split(qv[k].z, hi.z, lo.z);
                split(qv[k].w, hi.w, lo.w);
                uint8_t* dst = smem + (c / 8) * (2 * Rp * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
                *reinterpret_cast<uint4*>(dst) = hi;
                *reinterpret_cast<uint4*>(dst + Rp * 128) = lo;
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(QF);
            bar_128(bar_id);  // the row data
            float l[CW];
#pragma unroll
            for (int c = 0; c < CW; ++c) l[c] = 0.f;
            const uint32_t past = d[kPast];
            uint32_t place = d[kPlace];
            for (uint32_t left = d[kTiles]; left; --left, ++gt, place -= C::KT) {
                ok = warp_wait(SF, gt & 1) && ok;
                if (8u * sg >= Rp) {  // no rows for this warpgroup (which has to stay in step all the same)
                    if (lane == 0) mbar_arrive(SE);
                    if (gt) ok = warp_wait(PE + 8 * wq, (gt - 1) & 1) && ok;
                    if (lane == 0) mbar_arrive(PF + 8 * wq);
                    continue;
                }
                tc::fence_after_sync();
                float x[CW];
#pragma unroll
                for (int c = 0; c < CW; c += 8) {
                    uint32_t a[8] = {}, b[8] = {};
                    const uint32_t col = 4 * c + 8 * sg;
                    if (col < Rp) {
                        tc::tmem_ld8(tlane + C::C_S + col, a);
                        tc::tmem_ld8(tlane + C::C_S + Rp + col, b);
                        tc::tmem_ld_wait();
                    }
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const float2 y = join2(make_float2(__uint_as_float(a[k]), __uint_as_float(a[k + 1])),
                                               make_float2(__uint_as_float(b[k]), __uint_as_float(b[k + 1])),
                                               C::UNCUT_S);
                        x[c + k] = y.x;
                        x[c + k + 1] = y.y;
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(SE);
                // whether the tile has keys that some row does not attend: nodes, or what
                // the rule leaves out
                bool masked = place + C::KT > past;
                uint32_t on = 0xffffffffu;  // a bit per row: this thread's key is attended
                uint32_t kp = place + key;   // the key's place, then its position
                if (masked && kp >= past) {
                    const uint32_t j = kp - past;
                    on = 0u;
                    if (j < d[kNodes]) {
                        if (SC) kp = past + P.depth[d[kRow] + j];
                        // the nodes that attend this one, from the block's first (at most 64 of them)
                        const uint32_t n0 = d[kRow0] / G, w0 = n0 / 32;
                        const uint32_t* below = P.below + static_cast<size_t>(d[kRow] + j) * kTreeWords;
                        const uint32_t a = below[w0], b = w0 + 1 < kTreeWords ? below[w0 + 1] : 0u;
                        const uint32_t c2 = w0 + 2 < kTreeWords ? below[w0 + 2] : 0u;
                        const uint32_t lo = __funnelshift_r(a, b, n0 % 32), hi = __funnelshift_r(b, c2, n0 % 32);
#pragma unroll
                        for (int c = 0; c < CW; ++c) {
                            const uint32_t i = noder[32 * (c / 8) + c % 8];
                            on |= ((i < 32 ? lo : hi) >> (i % 32) & 1u) << c;
                        }
                    }
                }
                if constexpr (SC) {
                    if (P.rule.cap_out != 0.f) cap_scores<CW>(x, P.rule, cap_series(P.rule.cap_in));
                    const uint32_t window = P.rule.window;
                    const bool early = P.rule.doc_start && kp < __ldg(P.rule.doc_start + d[kReq]);
                    if (window || P.rule.doc_start) masked = true;
#pragma unroll
                    for (int c = 0; c < CW; c += 4) {
                        const int at = 32 * (c / 8) + c % 8;
                        const float4 sl = *reinterpret_cast<const float4*>(sloper + at);
                        const uint4 ps = *reinterpret_cast<const uint4*>(posr + at);
                        const uint32_t far[4] = {ps.x - kp, ps.y - kp, ps.z - kp, ps.w - kp};
                        const float by[4] = {sl.x, sl.y, sl.z, sl.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            x[c + k] = fmaf(-by[k], static_cast<float>(static_cast<int>(far[k])), x[c + k]);
                            if (early || (window && far[k] >= window)) on &= ~(1u << (c + k));
                        }
                    }
                }
                if (masked) {
#pragma unroll
                    for (int c = 0; c < CW; ++c) x[c] = on >> c & 1u ? x[c] : -CUDART_INF_F;
                }
                float over[2] = {-1e30f, -1e30f};  // by how much the scores pass the maxima
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(ms + 32 * (c / 8) + c % 8);
                    const float2 y = sub2(make_float2(x[c], x[c + 1]), make_float2(m.x, m.y));
                    const float2 z = sub2(make_float2(x[c + 2], x[c + 3]), make_float2(m.z, m.w));
                    over[0] = fmaxf(over[0], fmaxf(y.x, y.y));
                    over[1] = fmaxf(over[1], fmaxf(z.x, z.y));
                }
                if (bar_or(bar_id, fmaxf(over[0], over[1]) > 8.f)) {
                    // every row's maximum over the tile (as integers in the same order); the
                    // accumulators have read the last factors, and are done with the last unit.
                    // (P V of a tile starts when the one before it has been added, so behind PE's
                    // phase FX is at its last one)
                    if (gt) ok = warp_wait(PE + 8 * wq, (gt - 1) & 1) && warp_wait(FX, (gt - 1) & 1) && ok;
                    if (u && left == d[kTiles]) ok = warp_wait(UE, (u - 1) & 1) && ok;
#pragma unroll
                    for (int c = 0; c < CW; ++c) {
                        const int b = __float_as_int(x[c] == x[c] ? x[c] : -1e30f);
                        const int top = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
                        if (lane == 0) tmax[wq * RB + row_of(c)] = __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
                    }
                    bar_128(bar_id);
                    if (key < CW) {
                        const int row = row_of(key), at = row - 8 * sg;
                        const float top = fmaxf(fmaxf(tmax[row], tmax[RB + row]),
                                                fmaxf(tmax[2 * RB + row], tmax[3 * RB + row]));
                        const float old = ms[at], m = fmaxf(old, top);
                        // (not 0: an infinity that the row holds has to stay one)
                        fs[at] = fmaxf(tree_exp2(old - m), 1.17549435e-38f);
                        ms[at] = m;
                        if (key == 0) misc[12 + sg] = gt + 1;
                    }
                    bar_128(bar_id);
#pragma unroll
                    for (int c = 0; c < CW; ++c) l[c] *= fs[32 * (c / 8) + c % 8];
                }
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(ms + 32 * (c / 8) + c % 8);
                    const float2 y = sub2(make_float2(x[c], x[c + 1]), make_float2(m.x, m.y));
                    const float2 z = sub2(make_float2(x[c + 2], x[c + 3]), make_float2(m.z, m.w));
                    x[c] = tree_exp2(y.x);
                    x[c + 1] = tree_exp2(y.y);
                    x[c + 2] = tree_exp2(z.x);
                    x[c + 3] = tree_exp2(z.y);
                }
                if (masked) {  // the accumulators tell a masked key by its sign
#pragma unroll
                    for (int c = 0; c < CW; ++c) x[c] = on >> c & 1u ? x[c] : -0.f;
                }
#pragma unroll
                for (int c = 0; c < CW; c += 2) {
                    const float2 y = add2(make_float2(l[c], l[c + 1]), make_float2(x[c], x[c + 1]));
                    l[c] = y.x;
                    l[c + 1] = y.y;
                }
                // this warp's block of P is free once the MMAs have read the last tile's (and, where V
                // was not finite there, the accumulators have); at a unit's start, once the
                // accumulators are done with the last unit
                if (gt) {
                    ok = warp_wait(PE + 8 * wq, (gt - 1) & 1) && ok;
                    if (misc[4 + 4 * ((gt - 1) & 1) + wq] == gt) ok = warp_wait(FX, (gt - 1) & 1) && ok;
                    if (u && left == d[kTiles]) ok = warp_wait(UE, (u - 1) & 1) && ok;
                }
                // P^T: [32-key blocks][hi rows | lo rows][128 B], 16-byte pieces swizzled by the row
                const uint32_t dst = sbase + C::OFF_P + wq * (2 * Rp * 128) + 8 * sg * 128 + (lane >> 2) * 16 +
                                     (lane & 3) * 4;
                const uint32_t dst2 = dst + Rp * 128;
#pragma unroll
                for (int c = 0; c < CW; c += 2) {
                    if (4 * (c / 8 * 8) + 8 * sg < static_cast<int>(Rp)) {
                        const float2 hi = near2(x[c], x[c + 1]);
                        const float2 lo = sub2(make_float2(x[c], x[c + 1]), make_float2(__uint_as_float(tf32_part(hi.x)),
                                                                                       __uint_as_float(tf32_part(hi.y))));
                        const int at = (32 * (c / 8) + c % 8) * 128;
                        sts(dst ^ (c % 8) << 4, at, hi.x);
                        sts(dst2 ^ (c % 8) << 4, at, lo.x);
                        sts(dst ^ (c % 8 + 1) << 4, at + 128, hi.y);
                        sts(dst2 ^ (c % 8 + 1) << 4, at + 128, lo.y);
                    }
                }
                if (left == 1) {  // the rows' sums over the warp's keys, a lane per row
#pragma unroll
                    for (int off = 16; off >= CW; off >>= 1)
#pragma unroll
                        for (int c = 0; c < CW; ++c) l[c] += __shfl_xor_sync(0xffffffffu, l[c], off);
#pragma unroll
                    for (int h = CW / 2; h > 0; h >>= 1) {
                        const bool up = lane & h;
#pragma unroll
                        for (int c = 0; c < h; ++c) {
                            const float give = up ? l[c] : l[c + h], mine = up ? l[c + h] : l[c];
                            l[c] = mine + __shfl_xor_sync(0xffffffffu, give, h);
                        }
                    }
                    if (lane < CW) tmax[wq * RB + row_of(lane)] = l[0];
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(PF + 8 * wq);
            }
            done(u);
        }
    } else if (warp < 20) {
        // ------------------------------------------------------------ accumulators
        regs_increase<kRegAcc>();
        grid_dependency_wait();
        const int w = warp & 3, me = w * 32 + lane;
        const uint32_t tlane = tb + (static_cast<uint32_t>(w) << 21);
        float* fs = reinterpret_cast<float*>(smem + C::OFF_F);
        const float* sums = reinterpret_cast<const float*>(smem + C::OFF_MAX);
        const float uncut = C::FOLD && me >= 64 ? C::UNCUT_V : 1.f;  // (FOLD: V's low parts have lanes of their own)
        bool ok = true;
        uint32_t gt = 0;
        for (uint32_t u = 0;; ++u) {
            ok = known(u) && ok;
            const volatile uint32_t* d = words(u);
            if (bar_or(5, !ok || !d[kMore])) break;
            const uint32_t rows = d[kRows], Rp = (rows + 15) / 16 * 16;
            float o[C::DH][RB];
#pragma unroll
            for (int h = 0; h < C::DH; ++h)
#pragma unroll
                for (int c = 0; c < RB; ++c) o[h][c] = 0.f;
            uint32_t place = d[kPlace];
            for (uint32_t left = d[kTiles]; left; --left, ++gt, place -= C::KT) {
                ok = warp_wait(OF, gt & 1) && ok;
                tc::fence_after_sync();
                // (all tags at once: beside the MMAs each load takes 200 cycles)
                const uint4 raised = lds4(sbase + C::OFF_MISC + 48), odd = lds4(sbase + C::OFF_MISC + 16 + 16 * (gt & 1));
                if (raised.x == gt + 1 || raised.y == gt + 1 || raised.z == gt + 1 || raised.w == gt + 1) {
#pragma unroll
                    for (int sg = 0; sg < 4; ++sg) {
                        // the maxima were raised: what there is shrinks
                        if ((sg == 0 ? raised.x : sg == 1 ? raised.y : sg == 2 ? raised.z : raised.w) != gt + 1) continue;
#pragma unroll
                        for (int c = 0; c < RB; ++c) {
                            if ((c / 8) % 4 != sg) continue;
                            const float f = fs[c];
#pragma unroll
                            for (int h = 0; h < C::DH; ++h) o[h][c] *= f;
                        }
                    }
                }
                // V values that are not finite
                const bool any = odd.x == gt + 1 || odd.y == gt + 1 || odd.z == gt + 1 || odd.w == gt + 1;
                for (uint32_t kb = any && !(C::FOLD && me >= C::VD) ? 0 : 4; kb < 4; ++kb) {
                    if (misc[4 + 4 * (gt & 1) + kb] != gt + 1) continue;
                    const uint32_t k0 = place + 32 * kb, end = d[kPast] + d[kNodes];
                    for (uint32_t k = 0; k < 32 && k0 + k < end; ++k) {
                        const size_t key = tree_place(P, d[kReq], k0 + k);
                        const size_t at = (key * P.n_kv_head + d[kKvHead]) * HD;
#pragma unroll
                        for (int h = 0; h < C::DH; ++h) {
                            const float v = P.V[at + h * C::VD + me];
                            if ((__float_as_uint(v) & 0x7F800000u) != 0x7F800000u) continue;
#pragma unroll
                            for (int c = 0; c < RB; ++c) {
                                if (c >= static_cast<int>(rows)) break;
                                const uint32_t p = *reinterpret_cast<const uint32_t*>(
                                    smem + C::OFF_P + kb * (2 * Rp * 128) + c * 128 +
                                    (((k / 4) ^ (c & 7)) << 4) + (k & 3) * 4);
                                if (p != 0x80000000u) o[h][c] += v;
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(FX);
#pragma unroll
                for (int h = 0; h < C::DH; ++h) {
#pragma unroll
                    for (int c = 0; c < RB / 16; ++c) {
                        if (c * 16 >= static_cast<int>(Rp)) break;
                        uint32_t a[16], b[16];
                        tc::tmem_ld16(tlane + C::C_O + h * 2 * RB + 16 * c, a);
                        tc::tmem_ld16(tlane + C::C_O + h * 2 * RB + Rp + 16 * c, b);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            const float2 hi = make_float2(__uint_as_float(a[k]), __uint_as_float(a[k + 1]));
                            const float2 lo = make_float2(__uint_as_float(b[k]), __uint_as_float(b[k + 1]));
                            const float2 was = make_float2(o[h][16 * c + k], o[h][16 * c + k + 1]);
                            const float2 y = C::FOLD ? join2(add2(hi, lo), was, uncut) : add2(join2(lo, hi, C::UNCUT_V), was);
                            o[h][16 * c + k] = y.x;
                            o[h][16 * c + k + 1] = y.y;
                        }
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(OE);
            }
            // the unit's end: O through P's buffer (at head dim 64 with the products of V's low
            // parts beside it), then a factor for every row, and out or the partial result
            float* stage = reinterpret_cast<float*>(smem + C::OFF_P);
            const bool write = !bar_or(5, !ok || misc[0] != 0u) && P.req_of[d[kRow]] == d[kReq];
#pragma unroll
            for (int h = 0; h < C::DH; ++h)
#pragma unroll
                for (int c = 0; c < RB; ++c)
                    stage[(C::FOLD && me >= 64 ? RB * 64 : 0) + c * HD + (C::FOLD ? me & 63 : h * C::VD + me)] = o[h][c];
            const bool whole = d[kWhole] != 0;
            const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + d[kStart];
            if (me < static_cast<int>(rows)) {
                float den = (sums[me] + sums[RB + me]) + (sums[2 * RB + me] + sums[3 * RB + me]), f = 1.f;
                const float m = reinterpret_cast<const float*>(smem + C::OFF_M)[(u & 1) * RB + me];
                if (whole) {
                    if (P.sinks)
                        den += tree_exp2(__ldg(P.sinks + d[kKvHead] * G + (d[kRow0] + me) % G) * kRuleLog2e - m);
                    f = den == 0.f ? 0.f : 1.f / den;
                } else if (write) {
                    *reinterpret_cast<float2*>(P.part_ml + 2 * (slot * RB + me)) = make_float2(m, den);
                }
                fs[me] = f;
            }
            bar_128(5);
            if (write) {
                constexpr int F4 = HD / 4;
                for (uint32_t i = me; i < rows * F4; i += 128) {
                    const uint32_t c = i / F4, at = d[kRow0] + c;
                    float4 x = reinterpret_cast<const float4*>(stage)[i];
                    if (C::FOLD) {
                        const float4 y = reinterpret_cast<const float4*>(stage + RB * 64)[i];
                        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                    }
                    const float f = fs[c];
                    x = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
                    const size_t row = (static_cast<size_t>(d[kRow] + at / G)) * P.n_head + d[kKvHead] * G + at % G;
                    *reinterpret_cast<float4*>((whole ? P.out + row * HD : P.part + (slot * RB + c) * HD) + i % F4 * 4) = x;
                }
            }
            bar_128(5);  // everyone has read the sums, the maxima, the factors and the rows ...
            if (lane == 0) mbar_arrive(UE);  // ... which are the next unit's from here on
            done(u);
        }
    } else if (warp < 28) {
        // ------------------------------------------------------------ converters
        // The two warpgroups take the pieces by turns; with an even number of
        // slots, of a tile's pieces and of buffers, each sees every phase of its
        // own barriers.  Pieces go round the buffers in order, K's and V's alike, so
        // a warpgroup fills one buffer while the MMAs read its other one.
        static_assert(NSLOT % 2 == 0 && C::KP % 2 == 0 && C::VP % 2 == 0 && C::NB == 4, "turns");
        regs_decrease<kRegConv>();
        const uint32_t turn = warp < 24 ? 0u : 1u;
        const int w = warp & 3, me = w * 32 + lane;
        const uint32_t tlane = tb + (static_cast<uint32_t>(w) << 21);
        // this warpgroup's slot and the parity of its piece, its buffer and the parity of that
        // being empty, tiles
        uint32_t sl = turn, phase = 0, buf = turn, empty = 1, gt = 0;
        bool ok = true;
        for (uint32_t u = 0;; ++u) {
            ok = known(u) && ok;
            const volatile uint32_t* d = words(u);
            if (!ok || !d[kMore]) break;
            const uint32_t last = 2 * d[kTiles] - 1;
            uint32_t end = d[kPast] + d[kNodes] - d[kPlace];  // keys that the request has from the tile on
            // A piece's stores to tensor memory are waited for, and the piece handed over, only
            // after the next piece's loads, if that has landed already.
            uint32_t handed = 0;  // the barrier of the piece that is still to be handed over
            auto hand_over = [&]() {
                if (!handed) return;
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(handed);
                handed = 0;
            };
            auto landed = [&]() {
                if (__all_sync(0xffffffffu, mbar_test(RF + 8 * sl, phase))) return;
                hand_over();
                ok = warp_wait(RF + 8 * sl, phase) && ok;
            };
            auto read = [&]() {  // the slot is free; to the next one
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(RE + 8 * sl);
                sl += 2;
                if (sl >= NSLOT) sl = turn, phase ^= 1;
            };
            // the piece's stores are on their way; the next one goes into the other buffer
            auto stored = [&](uint32_t full) {
                read();
                handed = full + 8 * buf;
                buf ^= 2;
                if (buf == turn) empty ^= 1;
            };
            // K(0), then K(t + 1) and V(t) by turns
            for (uint32_t i = 0; i <= last; ++i) {
                if (i == last || (i && !(i & 1))) {
#pragma unroll 1
                    for (int j = static_cast<int>(turn); j < C::VP; j += 2) {
                        landed();
                        const float* src = reinterpret_cast<const float*>(smem + C::OFF_RING + sl * C::PIECE) + me % C::VD;
                        const uint32_t dst = tlane + C::C_B + C::BCOLS * buf;
#pragma unroll 1
                        for (int h = 0; h < C::VK / 32; ++h) {  // 32 keys at a time
                            const uint32_t k0 = j / C::DH * C::VK + 32 * h;
                            uint32_t x[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(src[(32 * h + k) * C::VD]);
                            if (k0 + 32 > end) {
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    if (k0 + k >= end) x[k] = 0u;
                            }
                            if (h == 0) {
                                hand_over();
                                ok = warp_wait(BE + 8 * buf, empty) && ok;
                                tc::fence_after_sync();
                            }
                            // the landed values are their own high parts
                            if (!C::FOLD || w < 2) tc::tmem_st32(dst + 32 * h, x);
                            float2 sum = make_float2(0.f, 0.f);  // of the low parts: NaN where a value is not finite
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                const float2 lo = low2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                                sum = add2(sum, lo);
                                x[k] = __float_as_uint(lo.x);
                                x[k + 1] = __float_as_uint(lo.y);
                            }
                            if (!C::FOLD || w >= 2) tc::tmem_st32((C::FOLD ? dst : dst + 32) + 32 * h, x);
                            if (__any_sync(0xffffffffu, !(sum.x + sum.y == sum.x + sum.y))) {
                                // such values are zeros to the tensor core; once more
                                if (lane == 0) misc[4 + 4 * (gt & 1) + k0 / 32] = gt + 1;
                                tc::tmem_st_wait();
#pragma unroll 1
                                for (int low = 0; low < 2; ++low) {
#pragma unroll
                                    for (int k = 0; k < 32; ++k) {
                                        const float v = src[(32 * h + k) * C::VD];
                                        x[k] = k0 + k >= end || (__float_as_uint(v) & 0x7F800000u) == 0x7F800000u
                                                   ? 0u
                                                   : low ? __float_as_uint(v - __uint_as_float(tf32_part(v)))
                                                         : __float_as_uint(v);
                                    }
                                    if (!C::FOLD)
                                        tc::tmem_st32(dst + 32 * low, x);
                                    else if ((w >= 2) == (low != 0))
                                        tc::tmem_st32(dst + 32 * h, x);
                                }
                            }
                        }
                        stored(VF);
                    }
                    ++gt;
                    end += C::KT;
                } else {
#pragma unroll 1
                    for (int j = static_cast<int>(turn); j < C::KP; j += 2) {
                        landed();
                        const uint8_t* src = smem + C::OFF_RING + sl * C::PIECE + me * 128;
                        uint32_t x[32];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint4 y = *reinterpret_cast<const uint4*>(src + ((c ^ (me & 7)) << 4));
                            x[4 * c] = y.x;
                            x[4 * c + 1] = y.y;
                            x[4 * c + 2] = y.z;
                            x[4 * c + 3] = y.w;
                        }
                        hand_over();
                        ok = warp_wait(BE + 8 * buf, empty) && ok;
                        tc::fence_after_sync();
                        const uint32_t dst = tlane + C::C_B + C::BCOLS * buf;
                        tc::tmem_st32(dst, x);  // (the landed values are their own high parts)
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float2 lo = low2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                            x[k] = __float_as_uint(lo.x);
                            x[k + 1] = __float_as_uint(lo.y);
                        }
                        tc::tmem_st32(dst + 32, x);
                        stored(KF);
                    }
                }
            }
            hand_over();
            done(u);
        }
    } else if (warp == 28) {
        // ------------------------------------------------------------ producer
        regs_decrease<kRegAux>();
        grid_dependency_wait();
        bool ok = true;
        uint32_t sl = 0, phase = 1, sent = 0;  // the slot, the parity of its being empty, pieces sent
        const uint32_t box = P.box_keys, lb = 31 - __clz(box), boxes = C::KT >> lb;
        const uint32_t vbox = min(box, static_cast<uint32_t>(C::VK)), vboxes = max(C::VK >> lb, 1);
        for (uint32_t u = 0;; ++u) {
            ok = known(u) && ok;
            const volatile uint32_t* d = words(u);
            if (!ok || !d[kMore]) break;
            const uint32_t last = 2 * d[kTiles] - 1, x0 = d[kKvHead] * HD, end = d[kPast] + d[kNodes];
            const uint32_t r = d[kReq];
            uint32_t place = d[kPlace];
            // the row of this lane's box of the tile at p
            auto row_at = [&](uint32_t p) {
                const uint32_t k = p + lane * box;
                return static_cast<uint32_t>(lane) < boxes && k < end ? tree_place(P, r, k) : 0u;
            };
            uint32_t yv = 0, yk = 0, next = row_at(place);  // the tiles of V, of K, and the next one's
            // K(0), then K(t + 1) and V(t) by turns
#pragma unroll 1
            for (uint32_t i = 0; i <= last; ++i) {
                const bool v = i == last || (i && !(i & 1));
                if (!v) {
                    yv = yk;
                    yk = next;
                    place -= C::KT;
                    if (i + (i ? 2 : 1) < last) next = row_at(place);
                }
                // this lane's box of the first piece: its key, and what there is of it
                uint32_t k = lane * (v ? vbox : box), x = x0;
                const uint32_t y = !v || i == last ? yk : yv, off = sbase + C::OFF_RING + k * (v ? C::VD * 4 : 128);
                const bool mine = static_cast<uint32_t>(lane) < (v ? vboxes : boxes);
                const CUtensorMap* map = v ? &tmV : &tmK;
                static_assert(C::KP == C::VP, "pieces");
#pragma unroll 1
                for (int j = 0; j < C::KP; ++j) {
                    const uint32_t row = __shfl_sync(0xffffffffu, y, k >> lb & 31) + (k & (box - 1));
                    ok = ok && warp_wait(RE + 8 * sl, phase);
                    if (!ok) break;
                    if (lane == 0) mbar_expect_tx(RF + 8 * sl, C::PIECE);
                    __syncwarp();
                    if (mine)
                        tma_load_2d(off + sl * C::PIECE, map, static_cast<int>(x), static_cast<int>(row), RF + 8 * sl);
                    ++sent;
                    if (++sl == NSLOT) sl = 0, phase ^= 1;
                    if (!v) {
                        x += 32;
                    } else if (C::DH == 1 || (j & 1)) {
                        k += C::VK;
                        x = x0;
                    } else {
                        x += C::VD;
                    }
                }
            }
            done(u);
        }
        grid_launch_dependents();
        if (misc[0])  // copies that may still be in flight
            for (uint32_t s = 0; s < NSLOT && s < sent; ++s)
                mbar_wait(RF + 8 * s, (sent - 1 - s) / NSLOT & 1, 1ll << 28);
    } else if (warp == 31) {
        // ------------------------------------------------------------ units
        regs_decrease<kRegAux>();
        // the prep kernel's plan says where this CTA's part begins
        grid_dependency_wait();
        const uint4* from = reinterpret_cast<const uint4*>(P.plan + kTreePlan * static_cast<size_t>(blockIdx.x));
        uint32_t d[kTreePlan];
#pragma unroll
        for (uint32_t i = 0; i < kTreePlan / 4; ++i) {
            const uint4 x = __ldcg(from + i);
            d[4 * i] = x.x;
            d[4 * i + 1] = x.y;
            d[4 * i + 2] = x.z;
            d[4 * i + 3] = x.w;
        }
        auto wide = [&](int i) { return static_cast<uint64_t>(d[i + 1]) << 32 | d[i]; };
        TreeWalk<RB> walk;
        walk.known = false;
        walk.k = static_cast<int>(d[kPlanSize]);
        walk.member = d[kPlanMember];
        walk.r = d[kPlanReq];
        walk.off = wide(kPlanOff);
        walk.left = wide(kPlanLeft);
        const uint64_t u1 = wide(kPlanEnd), each = wide(kPlanEach);
        const uint32_t over = d[kPlanOver];
        uint32_t unit_tiles = d[kPlanUnitTiles], u[12];
#pragma unroll
        for (int i = 0; i < 12; ++i) u[i] = d[i];
        // (the swizzled tiles need the 1 KB alignment that dynamic shared memory starts at)
        if (sbase & 1023u) {
            u[kMore] = 0u;
            misc[0] = 1;
        }
        // nothing for the combine kernel to join from here on, unless there turns out to be
        uint32_t* join = P.join + kTreeJoin * blockIdx.x;
        if (lane == 0) join[kJoinRows] = join[kJoinGaveUp] = 0u;
        for (uint32_t n = 0;; ++n) {
            if (n >= 2 && !warp_wait(GE + 8 * (n & 1), ((n >> 1) - 1) & 1)) break;
            if (lane == 0) {
                volatile uint32_t* to = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_DESC) + 12 * (n & 1);
                if (u[kMore])
#pragma unroll
                    for (int i = 0; i < 11; ++i) to[i] = u[i];
                to[kMore] = u[kMore];
                mbar_arrive(GF + 8 * (n & 1));
            }
            __syncwarp();
            if (!u[kMore]) break;
            if (u[kStart] && !u[kWhole] && lane == 0) {  // (the CTA's last; ends in another one)
                const uint64_t first_tile = u1 - u[kTiles], last_tile = first_tile + unit_tiles - 1;
                join[kJoinTok] = u[kRow];
                join[kJoinRow0] = u[kRow0];
                join[kJoinRows] = u[kRows];
                join[kJoinKvHead] = u[kKvHead];
                join[kJoinReq] = u[kReq];
                join[kJoinStep] = 1u << walk.k;
                join[kJoinParts] = tree_owner(each, over, last_tile) - tree_owner(each, over, first_tile) + 1;
            }
            if (!walk.next(P, u)) u[kMore] = 0u;
            unit_tiles = walk.x.tl;
        }
    } else {
        // ------------------------------------------------------------ MMA issuers
        // Warp 29 issues the products of S, warp 30 those of P V: while one waits
        // at a barrier (a couple of hundred cycles beside MMAs that read shared
        // memory) the other's MMAs run.
        regs_decrease<kRegAux>();
        const bool lead = tc::elect_one();
        bool ok = true;
        uint32_t full = 0, tiles = 0;  // the parities of its pieces in the buffers, its tiles
        for (uint32_t u = 0;; ++u) {
            ok = known(u) && ok;
            const volatile uint32_t* d = words(u);
            // (the same in all lanes, so that an MMA's operands are in uniform registers)
            if (!ok || !__shfl_sync(0xffffffffu, d[kMore], 0)) break;
            const uint32_t Rp = __shfl_sync(0xffffffffu, (d[kRows] + 15) / 16 * 16, 0);
            const uint32_t n = __shfl_sync(0xffffffffu, d[kTiles], 0);
            done(u);
            const uint32_t i2 = tc::idesc_tf32(128, 0, false) | (2 * Rp >> 3) << 17;
            const uint32_t i1 = tc::idesc_tf32(128, 0, false) | (Rp >> 3) << 17;
            const uint32_t block = 2 * Rp * 128 >> 4;  // a 32-wide block of Q or P
            if (warp == 29) {
                const uint64_t qdesc0 = tc::smem_desc(sbase, 16, 1024, tc::kSwizzle128B);
                const uint32_t sc = tb + C::C_S, sl2 = sc + Rp;
                ok = warp_wait(QF, u & 1) && ok;
                for (uint32_t t = 0; t < n; ++t, ++tiles) {
                    if (tiles) ok = warp_wait(SE, (tiles - 1) & 1) && ok;
                    uint32_t b = t ? C::KP % C::NB : 0;  // K(t) comes behind 2 t - 1 others
#pragma unroll 1
                    for (int j = 0; j < C::KP; ++j, b = (b + 1) % C::NB) {
                        ok = warp_wait(KF + 8 * b, full >> b & 1) && ok;
                        full ^= 1u << b;
                        if (!ok) continue;
                        tc::fence_after_sync();
                        const uint64_t qd = qdesc0 + j * block;
                        const uint32_t k = tb + C::C_B + C::BCOLS * b, free = BE + 8 * b;
                        const uint32_t more = j ? 1u : 0u;
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc::mma_tf32_ts(sc, k + 8 * kk, qd + 2 * kk, i2, kk ? 1u : more);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                tc::mma_tf32_ts(sl2, k + 32 + 8 * kk, qd + 2 * kk, i1, 1u);
                            tc::mma_commit(free);
                        }
                        __syncwarp();
                    }
                    // (the failure-path test option withholds the CTA's first score-ready signal)
                    if (lead && ok && !(tiles == 0 && (P.flags & kOptTestStall))) tc::mma_commit(SF);
                    __syncwarp();
                }
            } else {
                const uint64_t pdesc0 = tc::smem_desc(sbase + C::OFF_P, 16, 1024, tc::kSwizzle128B);
                for (uint32_t t = 0; t < n; ++t, ++tiles) {
                    if (tiles) ok = warp_wait(OE, (tiles - 1) & 1) && ok;
                    uint32_t b = t == n - 1 ? C::VP % C::NB : 0;  // V(t) comes behind 2 t + 2, the last behind 2 n - 1
#pragma unroll 1
                    for (int j = 0; j < C::VP; ++j, b = (b + 1) % C::NB) {
                        if (j % C::DH == 0)
#pragma unroll
                            for (int h = 0; h < C::VK / 32; ++h)
                                ok = warp_wait(PF + 8 * (j / C::DH * (C::VK / 32) + h), tiles & 1) && ok;
                        ok = warp_wait(VF + 8 * b, full >> b & 1) && ok;
                        full ^= 1u << b;
                        if (!ok) continue;
                        tc::fence_after_sync();
                        const uint32_t a = tb + C::C_B + C::BCOLS * b, o = tb + C::C_O + j % C::DH * 2 * RB;
                        const uint32_t ol = o + Rp;
                        const uint64_t pd = pdesc0 + j / C::DH * (C::VK / 32) * block, pd2 = pd + block;
                        const uint32_t more = j >= C::DH ? 1u : 0u;
                        const uint32_t free = BE + 8 * b, pe = PE + 8 * (j / C::DH * (C::VK / 32));
                        const bool last = j % C::DH == C::DH - 1;
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < C::VK / 8; ++kk)
                                tc::mma_tf32_ts(o, a + 8 * kk, (kk < 4 ? pd : pd2) + 2 * (kk % 4), i2,
                                                kk ? 1u : more);
#pragma unroll
                            for (int kk = 0; kk < (C::FOLD ? 0 : 4); ++kk)
                                tc::mma_tf32_ts(ol, a + 32 + 8 * kk, pd + 2 * kk, i1, 1u);
                            tc::mma_commit(free);
                            if (last)
#pragma unroll
                                for (int h = 0; h < C::VK / 32; ++h) tc::mma_commit(pe + 8 * h);
                        }
                        __syncwarp();
                    }
                    if (lead && ok) tc::mma_commit(OF);
                    __syncwarp();
                }
            }
        }
        // every MMA has ended before tensor memory is freed
        const uint32_t drain = DRAIN + 8 * (warp - 29);
        if (lead) tc::mma_commit(drain);
        __syncwarp();
        mbar_wait(drain, 0);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 29) tc::tmem_dealloc(tb, C::TMEM_COLS);
    if (tid == 0 && misc[0]) {
        atomicOr(P.status, kDevTimeout);
        P.join[kTreeJoin * blockIdx.x + kJoinGaveUp] = 1u;
    }
}

// ------------------------------------------------------------------ combine
// The units that lie in several CTAs, of which there is one at most that begins in
// a CTA: its partial results in the CTAs' order, a warp per row.
//   m = max_i m_i,  out = sum_i O_i 2^(m_i - m) / (sum_i l_i 2^(m_i - m) + e^sink 2^-m)
// Three dependent loads and at most 2 x 152 x 64 rows; a warp for each of the call's
// rows, most of which have nothing to join, took 10 us more for 20 thousand rows.
constexpr int kJoinThreads = 256;
template <int HD>
__global__ void __launch_bounds__(kJoinThreads) slotkv_tree_combine_kernel(const TreeParams P) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int RB = TreeCfg<HD>::RB, E = HD / 32;
    const int lane = threadIdx.x & 31;
    const uint32_t row = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const uint4* join = reinterpret_cast<const uint4*>(P.join + kTreeJoin * blockIdx.x);
    const uint4 j0 = __ldcg(join), j1 = __ldcg(join + 1);
    const uint32_t rows = j0.z, step = j1.y, parts = j1.z;
    if (row >= rows) return;
    const uint32_t G = P.n_head / P.n_kv_head, at = j0.y + row;
    const uint32_t tok = j0.x + at / G, h = j0.w * G + at % G;
    // part i's row: the first CTA's last unit, the others' first one
    auto slot = [&](uint32_t i) {
        return (2 * static_cast<size_t>(blockIdx.x + i * step) + (i ? 0 : 1)) * RB + row;
    };
    // whether part i's CTA gave up
    auto gave_up = [&](uint32_t i) { return __ldcg(P.join + kTreeJoin * (blockIdx.x + i * step) + kJoinGaveUp); };
    float2 ml = make_float2(-1e30f, 0.f);
    uint32_t lost = 0;
    if (static_cast<uint32_t>(lane) < parts) {
        ml = __ldcg(reinterpret_cast<const float2*>(P.part_ml) + slot(lane));
        lost = gave_up(lane);
    }
    if (__ldcg(P.req_of + tok) != j1.x) return;  // (refused)
    float m = ml.x;
    for (uint32_t i = lane + 32; i < parts; i += 32) {
        m = fmaxf(m, __ldcg(P.part_ml + 2 * slot(i)));
        lost |= gave_up(i);
    }
    if (__any_sync(0xffffffffu, lost != 0u)) return;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float den = 0.f, acc[E] = {};
#pragma unroll 4
    for (uint32_t i = 0; i < parts; ++i) {
        if (i && i % 32 == 0)
            ml = i + lane < parts ? __ldcg(reinterpret_cast<const float2*>(P.part_ml) + slot(i + lane))
                                  : make_float2(-1e30f, 0.f);
        const float mi = __shfl_sync(0xffffffffu, ml.x, i % 32), li = __shfl_sync(0xffffffffu, ml.y, i % 32);
        const float f = fmaxf(tree_exp2(mi - m), 1.17549435e-38f);  // (see the raise)
        den = fmaf(li, f, den);
        const float* src = P.part + slot(i) * HD + lane;
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] = fmaf(__ldcg(src + 32 * j), f, acc[j]);
    }
    if (P.sinks) den += tree_exp2(__ldg(P.sinks + h) * kRuleLog2e - m);
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int j = 0; j < E; ++j) P.out[(static_cast<size_t>(tok) * P.n_head + h) * HD + lane + 32 * j] = acc[j] * inv;
}

template <int HD>
int launch_tree_hd(TreeParams p, const CUtensorMap& tmK, const CUtensorMap& tmV, uint32_t sms,
                   cudaStream_t stream) {
    using C = TreeCfg<HD>;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    cudaError_t e;
    if (!(configured.load(std::memory_order_acquire) & bit) || bit == 0) {
        const cudaFuncAttribute which = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if ((e = cudaFuncSetAttribute(slotkv_tree_attn_kernel<HD, false>, which, C::SMEM)) != cudaSuccess ||
            (e = cudaFuncSetAttribute(slotkv_tree_attn_kernel<HD, true>, which, C::SMEM)) != cudaSuccess)
            return static_cast<int>(e);
        // the register hand-over assumes what the kernels are launched with: with fewer the
        // softmax warps' request could never be met
        cudaFuncAttributes fa[2];
        if ((e = cudaFuncGetAttributes(&fa[0], slotkv_tree_attn_kernel<HD, false>)) != cudaSuccess ||
            (e = cudaFuncGetAttributes(&fa[1], slotkv_tree_attn_kernel<HD, true>)) != cudaSuccess)
            return static_cast<int>(e);
        if (fa[0].numRegs != kTreeRegs || fa[1].numRegs != kTreeRegs)
            return static_cast<int>(cudaErrorInvalidConfiguration);
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // parts: about one item per warp for requests of the mean size
    const uint64_t mean = (p.n_tok + p.n_req - 1) / p.n_req;
    uint64_t parts = 0;
    for (p.prep_heads = 1;; p.prep_heads *= 2) {
        const uint32_t kvh = (p.prep_heads + 1) / 2;
        const uint32_t groups = (p.n_head + p.prep_heads - 1) / p.prep_heads + (p.n_kv_head + kvh - 1) / kvh;
        parts = (mean * groups + kPrepWarps - 1) / kPrepWarps;
        if (p.prep_heads == kPrepHeads || p.n_req * (1 + parts) <= static_cast<uint64_t>(kPrepCtas) * sms) break;
    }
    cfg.gridDim = dim3(p.n_req + 1, 1 + static_cast<unsigned>(parts < 256 ? parts : 256));
    cfg.blockDim = dim3(kPrepThreads);
    cfg.dynamicSmemBytes = kPrepWarps * 2 * ((p.prep_heads + 1) / 2) * HD * 4;
    if ((e = cudaLaunchKernelEx(&cfg, slotkv_tree_prep_kernel<HD>, p)) != cudaSuccess) return static_cast<int>(e);
    cfg.gridDim = dim3(tree_grid(sms));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    const bool rule = p.rule.cap_out != 0.f || p.rule.window || p.rule.slopes || p.rule.doc_start;
    e = rule ? cudaLaunchKernelEx(&cfg, slotkv_tree_attn_kernel<HD, true>, tmK, tmV, p)
             : cudaLaunchKernelEx(&cfg, slotkv_tree_attn_kernel<HD, false>, tmK, tmV, p);
    if (e != cudaSuccess) return static_cast<int>(e);
    cfg.gridDim = dim3(tree_grid(sms), C::RB / (kJoinThreads / 32));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, slotkv_tree_combine_kernel<HD>, p));
}

}  // namespace slotkv
