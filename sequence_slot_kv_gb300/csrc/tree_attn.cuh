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
// CTA (request, part): checks the request, finds every node's ancestors and
// depth (pointer doubling over the tree in shared memory: each round joins a
// node's set with that of the node it points at and doubles the distance, so
// a chain of 256 takes 8 rounds), then forms its part of the request's
// vectors, one warp per (node, kTreeQHeads query heads or kTreeKvHeads kv
// heads): q' = RoPE(RMSnorm(q) w) scale log2(e) into the workspace, k' and v
// into the node's cache row, with the decode kernel's vector routines (so
// the same bits as a decode step's at that position).
constexpr int kTreeQHeads = 8, kTreeKvHeads = 4, kPrepThreads = 128, kPrepWarps = kPrepThreads / 32;

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
    const uint64_t cap = P.block_tables ? static_cast<uint64_t>(P.bt_stride) * P.slot_ctx : P.slot_ctx;
    q.ok = q.s0 <= s1 && s1 <= P.n_tok && q.n <= kTreeNodes && static_cast<uint64_t>(q.past) + q.n <= cap;
    if (!P.block_tables) q.ok = q.ok && __ldg(P.slots + r) < P.n_slots;
    return q;
}

template <int HD>
constexpr int tree_prep_smem() {
    return kPrepWarps * kTreeQHeads * HD * 4;
}

template <int HD>
__global__ void __launch_bounds__(kPrepThreads) slotkv_tree_prep_kernel(const TreeParams P) {
    extern __shared__ __align__(16) uint8_t prep_smem[];
    __shared__ uint32_t set[kTreeNodes][kTreeWords];
    __shared__ uint32_t jump[kTreeNodes], depth[kTreeNodes];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t r = blockIdx.x;
    TreeReq q = tree_request(P, r);
    if (q.n == 0) return;
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
#pragma unroll
            for (uint32_t w = 0; w < kTreeWords; ++w) set[i][w] = i / 32 == w ? 1u << (i % 32) : 0u;
        }
    }
    ok = __syncthreads_and(ok) != 0;
    if (!ok) {
        if (blockIdx.y == 0) {
            if (tid == 0) atomicOr(P.status, kDevRange);
            if (q.s0 + q.n <= P.n_tok && q.n <= P.n_tok)  // (no more than the rows there are)
                for (uint32_t i = tid; i < q.n; i += kPrepThreads) P.req_of[q.s0 + i] = kTreeSkip;
        }
        return;
    }
    constexpr int PER = kTreeNodes / kPrepThreads;
    const uint32_t words = (q.n + 31) / 32;
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
    if (blockIdx.y == 0) {
        for (uint32_t i = tid; i < q.n; i += kPrepThreads) {
            P.req_of[q.s0 + i] = r;
            P.depth[q.s0 + i] = depth[i];
#pragma unroll
            for (uint32_t w = 0; w < kTreeWords; ++w)
                P.anc[static_cast<size_t>(q.s0 + i) * kTreeWords + w] = set[i][w];
        }
    }
    const uint32_t qg = (P.n_head + kTreeQHeads - 1) / kTreeQHeads;
    const uint32_t groups = qg + (P.n_kv_head + kTreeKvHeads - 1) / kTreeKvHeads;
    const float w1 = (P.flags & kOptNormPlusOne) ? 1.0f : 0.0f;
    float* rows = reinterpret_cast<float*>(prep_smem) + warp * kTreeQHeads * HD;
    float* vrows = rows + kTreeKvHeads * HD;
    for (uint32_t it = blockIdx.y * kPrepWarps + warp; it < q.n * groups; it += gridDim.y * kPrepWarps) {
        const uint32_t i = it / groups, grp = it % groups, tok = q.s0 + i;
        const bool is_q = grp < qg;
        const uint32_t x0 = is_q ? grp * kTreeQHeads : (grp - qg) * kTreeKvHeads;
        const uint32_t left = (is_q ? P.n_head : P.n_kv_head) - x0, most = is_q ? kTreeQHeads : kTreeKvHeads;
        const uint32_t nx = left < most ? left : most;
        for (uint32_t x = 0; x < nx; ++x) {
            const float* src = is_q ? P.q + (static_cast<size_t>(tok) * P.n_head + x0 + x) * HD
                                    : P.k_new + (static_cast<size_t>(tok) * P.n_kv_head + x0 + x) * HD;
            const float* vsrc = P.v_new + (static_cast<size_t>(tok) * P.n_kv_head + x0 + x) * HD;
            for (int c = lane; c < HD / 4; c += 32) {
                tree_cp_async16(rows + x * HD + 4 * c, src + 4 * c);
                if (!is_q) tree_cp_async16(vrows + x * HD + 4 * c, vsrc + 4 * c);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        float cs[HD / 64], sn[HD / 64];
        warp_rope_angles<HD>(q.past + depth[i], P.inv_freq, cs, sn, lane);
        const size_t at = is_q ? 0 : (static_cast<size_t>(tree_row(P, r, q.past + i)) * P.n_kv_head + x0) * HD;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        for (uint32_t x = 0; x < nx; ++x) {
            if (is_q) {
                warp_norm_rope<HD>(rows + x * HD,
                                   P.q_rot + (static_cast<size_t>(tok) * P.n_head + x0 + x) * HD, P.q_norm_w,
                                   w1, P.scale_log2, P.eps, cs, sn, lane);
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
// f32 bits are read with the low 13 mantissa bits ignored, so a landed K tile is
// its own high part.  The other A operands come from tensor memory, where a
// warp's lanes are the operand's rows: K's low part is written there by the
// thread that owns the key, V^T by the thread that owns the dim, which makes the
// transposition free.  At head dim 64 one A holds V^T's high part in lanes 0-63
// and its low part in lanes 64-127, and one MMA forms all four products.
//
// Roles (14 warps):
//   0-3   softmax: a thread per key of the tile.  Q rows into shared memory at a
//         unit's start; then per tile S from tensor memory, the rule and the
//         masks, P^T (hi, lo) into shared memory.  The running maxima are raised
//         lazily (by 2^8), all 128 threads agreeing at a named barrier.
//   4-7   converters: K's low part and V^T (hi, lo) into tensor memory.
//   8-11  accumulators: a thread per dim.  Every tile's O^T starts anew in
//         tensor memory (its chain of sums is cut toward zero at each step) and
//         is added to registers with rounded adds; also the rows' sums, from P.
//         At the end out, or the unit's partial result.
//   12    producer: 16 KB pieces of K (128 keys x 32 dims, swizzled) and V by TMA
//         into a ring.  13: MMA issuer.
// The pieces go K(0), K(1), V(0), K(2), V(1), ...: S(t + 1) is formed while the
// softmax of tile t runs.
//
// The tiles of all units, in order, are cut into one equal range per CTA (every
// CTA finds its own from the lengths), so a unit may lie in several CTAs; each
// leaves (m, l, O) then, and slotkv_tree_combine_kernel joins them in CTA order.
//
// Keys past the request's last are zeros in V; a masked key's P is -0.  A V value
// that is not finite is a 0 to the tensor core, and the accumulators add it to
// the rows that attend its key (P not -0), so it reaches no other row.
//
// Every wait is bounded.  Where one runs out, its CTA raises SLOTKV_DEV_TIMEOUT
// and sets a flag that ends all its other waits at once; the roles go through
// the rest of their loops without doing anything, so they meet at their barriers
// and at the end as ever.
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
    static constexpr int NKL = 4, NV = 2;               // buffers of K lo and of V^T
    // tensor memory columns
    static constexpr int C_S = 0, C_O = 2 * RB, C_KL = C_O + DH * 2 * RB, C_V = C_KL + NKL * 32;
    static constexpr int VCOLS = 64;                    // a V^T buffer: hi | lo, 32 keys each (FOLD: 64 keys)
    static_assert(C_V + NV * VCOLS <= 512, "tensor memory");
    static constexpr int TMEM_COLS = 512;
    // shared memory behind the ring: row data, scratch of the maxima, barriers, flags
    static constexpr int OFF_M = OFF_RING + NSLOT * PIECE;      // running maxima [RB]
    static constexpr int OFF_F = OFF_M + RB * 4;                // factors of a raise [RB]
    static constexpr int OFF_L = OFF_F + RB * 4;                // sums [RB]
    static constexpr int OFF_POS = OFF_L + RB * 4;              // rows' positions [RB]
    static constexpr int OFF_LO = OFF_POS + RB * 4;             // rows' first position attended [RB]
    static constexpr int OFF_SLOPE = OFF_LO + RB * 4;           // rows' slopes [RB]
    static constexpr int OFF_MAX = OFF_SLOPE + RB * 4;          // tile maxima [4][RB]
    static constexpr int OFF_BAR = OFF_MAX + 4 * RB * 4;
    // full, K empty, V empty [NSLOT]; K lo full, empty [NKL]; V full, empty [NV]; S full, empty;
    // P full, empty; O full, empty; Q full; unit's end; drain
    static constexpr int NBAR = 3 * NSLOT + 2 * NKL + 2 * NV + 9;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 64;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(OFF_BAR % 8 == 0 && NSLOT >= 6, "layout");
};
constexpr int kTreeWarps = 14, kTreeThreads = 32 * kTreeWarps;

// A part of a unit: its rows, and its tiles [t0, t1) of tl, from absolute tile
// tile0 on.
struct TreeSeg {
    uint32_t r, s0, n, past, g, row0, rows, tile0, t0, t1, tl;
};

// A request's shape: row blocks, first tile, tiles; 0 blocks: nothing to do.
struct TreeShape {
    TreeReq q;
    uint32_t nb, tile0, tl;
    __device__ uint64_t tiles(uint32_t n_kv_head) const {
        return static_cast<uint64_t>(nb) * tl * n_kv_head;
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

// The CTAs that share `total` tiles, and the first tile of CTA c.
__device__ __forceinline__ uint32_t tree_ctas(uint64_t total, uint32_t grid) {
    return total < grid ? static_cast<uint32_t>(total) : grid;
}
__device__ __forceinline__ uint64_t tree_first(uint64_t total, uint32_t ctas, uint32_t c) {
    return total * c / ctas;
}
// The CTA of tile x.
__device__ __forceinline__ uint32_t tree_owner(uint64_t total, uint32_t ctas, uint64_t x) {
    return static_cast<uint32_t>(((x + 1) * ctas - 1) / total);
}

// A CTA's segments in order; every role walks them by itself.
template <int RB>
struct TreeWalk {
    uint32_t r;
    uint64_t off, left;  // tiles into request r, tiles left
    TreeShape x;
    bool known;
    __device__ bool next(const TreeParams& P, TreeSeg& s) {
        if (left == 0) return false;
        for (;;) {
            if (!known) {
                if (r >= P.n_req) return false;
                x = tree_shape<RB>(P, r);
                known = true;
            }
            if (off < x.tiles(P.n_kv_head)) break;
            off -= x.tiles(P.n_kv_head);
            ++r;
            known = false;
        }
        const uint32_t unit = static_cast<uint32_t>(off / x.tl);
        s.r = r;
        s.s0 = x.q.s0;
        s.n = x.q.n;
        s.past = x.q.past;
        s.g = unit / x.nb;
        s.row0 = unit % x.nb * RB;
        const uint32_t all = x.q.n * (P.n_head / P.n_kv_head) - s.row0;
        s.rows = all < RB ? all : RB;
        s.tile0 = x.tile0;
        s.tl = x.tl;
        s.t0 = static_cast<uint32_t>(off - static_cast<uint64_t>(unit) * x.tl);
        const uint64_t end = s.t0 + left;
        s.t1 = end < x.tl ? static_cast<uint32_t>(end) : x.tl;
        off += s.t1 - s.t0;
        left -= s.t1 - s.t0;
        return true;
    }
};

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
// x without its low 13 mantissa bits: what the tensor core reads of it.
__device__ __forceinline__ uint32_t tf32_part(float x) { return __float_as_uint(x) & 0xFFFFE000u; }

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
    // misc: [0] abort, [1] a raise comes with P, [2], [3] the last tile (even, odd; plus 1) with
    // a V value that is not finite, [4] tensor memory
    const uint32_t bar0 = sbase + C::OFF_BAR;
    const uint32_t FULL = bar0, KE = FULL + 8 * NSLOT, VE = KE + 8 * NSLOT, KLF = VE + 8 * NSLOT,
                   KLE = KLF + 8 * C::NKL, VF = KLE + 8 * C::NKL, VFE = VF + 8 * C::NV, SF = VFE + 8 * C::NV,
                   SE = SF + 8, PF = SE + 8, PE = PF + 8, OF = PE + 8, OE = OF + 8, QF = OE + 8, UE = QF + 8, DRAIN = UE + 8;
    if (tid == 0) {
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(FULL + 8 * i, 1);
            mbar_init(KE + 8 * i, 1);
            mbar_init(VE + 8 * i, 4);
        }
        for (int i = 0; i < C::NKL; ++i) {
            mbar_init(KLF + 8 * i, 4);
            mbar_init(KLE + 8 * i, 1);
        }
        for (int i = 0; i < C::NV; ++i) {
            mbar_init(VF + 8 * i, 4);
            mbar_init(VFE + 8 * i, 1);
        }
        mbar_init(SF, 1);
        mbar_init(SE, 4);
        mbar_init(PF, 4);
        mbar_init(PE, 5);
        mbar_init(OF, 1);
        mbar_init(OE, 4);
        mbar_init(QF, 4);
        mbar_init(UE, 4);
        mbar_init(DRAIN, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < 4; ++i) misc[i] = 0;
    }
    if (warp == 13) {
        tc::tmem_alloc(sbase + C::OFF_MISC + 16, C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    // this CTA's range: every thread sums a part of the requests, a scan finds the
    // request that the range begins in.  The ring is not in use yet.
    uint64_t* sums = reinterpret_cast<uint64_t*>(smem);
    uint64_t* found = sums + kTreeWarps;  // request, tiles into it
    const uint32_t per = (P.n_req + kTreeThreads - 1) / kTreeThreads;
    const uint32_t ra = tid * per < P.n_req ? tid * per : P.n_req;
    const uint32_t rb = ra + per < P.n_req ? ra + per : P.n_req;
    uint64_t mine = 0;
    for (uint32_t r = ra; r < rb; ++r) mine += tree_shape<RB>(P, r).tiles(P.n_kv_head);
    uint64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    uint64_t at = incl - mine, total = 0;
    for (int w = 0; w < kTreeWarps; ++w) {
        if (w < warp) at += sums[w];
        total += sums[w];
    }
    const uint32_t ctas = tree_ctas(total, gridDim.x);
    const uint64_t u0 = ctas ? tree_first(total, ctas, blockIdx.x) : 0;
    const uint64_t u1 = ctas ? tree_first(total, ctas, blockIdx.x + 1) : 0;
    // (the swizzled tiles need the 1 KB alignment that dynamic shared memory starts at)
    const bool work = blockIdx.x < ctas && (sbase & 1023u) == 0;
    if ((sbase & 1023u) && tid == 0) atomicOr(P.status, kDevTimeout);
    if (work && at <= u0 && u0 < at + mine) {
        uint64_t off = u0 - at;
        for (uint32_t r = ra; r < rb; ++r) {
            const uint64_t n = tree_shape<RB>(P, r).tiles(P.n_kv_head);
            if (off < n) {
                found[0] = r;
                found[1] = off;
                break;
            }
            off -= n;
        }
    }
    if (blockIdx.x == 0) {  // for the combine kernel: every request's first tile, and the sum
        uint64_t b = at;
        for (uint32_t r = ra; r < rb; ++r) {
            P.base[r] = b;
            b += tree_shape<RB>(P, r).tiles(P.n_kv_head);
        }
        if (tid == 0) P.base[P.n_req] = total;
    }
    __syncthreads();
    TreeWalk<RB> walk;
    walk.known = false;
    walk.r = work ? static_cast<uint32_t>(found[0]) : 0u;
    walk.off = work ? found[1] : 0u;
    walk.left = work ? u1 - u0 : 0u;
    const uint32_t tb = __shfl_sync(0xffffffffu, misc[4], 0);
    __syncthreads();  // (the scan's words are Q's from here on)

    // A bounded wait; once the CTA has given up every wait ends at once.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return true;
        const long long start = clock64();
        for (uint32_t it = 0; it < (1u << 26); ++it) {
            if (mbar_try_wait(bar, parity)) return true;
            if (misc[0]) return false;
            if (clock64() - start > (1ll << 31)) break;
        }
        misc[0] = 1;
        atomicOr(P.status, kDevTimeout);
        return false;
    };
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    const uint32_t G = P.n_head / P.n_kv_head;
    TreeSeg s;

    if (warp < 4) {
        // ------------------------------------------------------------ softmax
        grid_dependency_wait();
        float* ms = reinterpret_cast<float*>(smem + C::OFF_M);
        float* fs = reinterpret_cast<float*>(smem + C::OFF_F);
        float* tmax = reinterpret_cast<float*>(smem + C::OFF_MAX);
        uint32_t* posr = reinterpret_cast<uint32_t*>(smem + C::OFF_POS);
        uint32_t* lor = reinterpret_cast<uint32_t*>(smem + C::OFF_LO);
        float* sloper = reinterpret_cast<float*>(smem + C::OFF_SLOPE);
        const CapSeries series = cap_series(P.rule.cap_in);
        const uint32_t tlane = tb + (static_cast<uint32_t>(warp) << 21);
        const int key = tid;  // of the tile
        bool ok = true;
        uint32_t gt = 0;  // tiles so far
        for (uint32_t units = 0; walk.next(P, s); ++units) {
            const uint32_t Rp = (s.rows + 15) / 16 * 16;
            // the accumulators are done with the unit before: its maxima, and P's buffer
            if (units) ok = warp_wait(UE, (units - 1) & 1) && warp_wait(PE, (gt - 1) & 1) && ok;
            if (tid < RB) {
                ms[tid] = -1e30f;
                const uint32_t row = tid < static_cast<int>(s.rows) ? tid : s.rows - 1;
                const uint32_t node = (s.row0 + row) / G, h = s.g * G + (s.row0 + row) % G;
                const uint32_t pos = s.past + P.depth[s.s0 + node];
                posr[tid] = pos;
                lor[tid] = SC ? rule_first(P.rule, s.r, pos) : 0u;
                sloper[tid] = SC && P.rule.slopes ? __ldg(P.rule.slopes + h) * kRuleLog2e : 0.f;
            }
            // Q rows, split with rounded high parts: [32-dim blocks][hi rows | lo rows][128 B]
            constexpr int F4 = HD / 4;  // float4s of a row
            for (uint32_t i0 = 0; i0 < Rp * F4; i0 += 8 * 128) {
                float4 x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t i = i0 + k * 128 + tid, row = i / F4, c = i % F4;
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (row < s.rows) {
                        const uint32_t node = (s.row0 + row) / G, h = s.g * G + (s.row0 + row) % G;
                        x[k] = *reinterpret_cast<const float4*>(
                            P.q_rot + (static_cast<size_t>(s.s0 + node) * P.n_head + h) * HD + 4 * c);
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t i = i0 + k * 128 + tid, row = i / F4, c = i % F4;
                    if (row >= Rp) continue;
                    uint4 hi, lo;
                    auto split = [](float v, uint32_t& a, uint32_t& b) {
                        a = (__float_as_uint(v) + 0x1000u) & 0xFFFFE000u;
                        b = __float_as_uint(v - __uint_as_float(a));
                    };
                    split(x[k].x, hi.x, lo.x);
                    split(x[k].y, hi.y, lo.y);
                    split(x[k].z, hi.z, lo.z);
                    split(x[k].w, hi.w, lo.w);
                    uint8_t* dst = smem + (c / 8) * (2 * Rp * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4*>(dst) = hi;
                    *reinterpret_cast<uint4*>(dst + Rp * 128) = lo;
                }
            }
            tc::fence_proxy_async_smem();
            bar_128(1);  // (the rows' data too)
            if (lane == 0) mbar_arrive(QF);
            for (uint32_t t = s.t0; t < s.t1; ++t, ++gt) {
                ok = warp_wait(SF, gt & 1) && ok;
                tc::fence_after_sync();
                float x[RB];
#pragma unroll
                for (int c = 0; c < RB / 16; ++c) {
                    if (c * 16 >= static_cast<int>(Rp)) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[16 * c + k] = 0.f;
                        continue;
                    }
                    uint32_t a[16], b[16];
                    tc::tmem_ld16(tlane + C::C_S + 16 * c, a);
                    tc::tmem_ld16(tlane + C::C_S + Rp + 16 * c, b);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[16 * c + k] = __uint_as_float(a[k]) + __uint_as_float(b[k]);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(SE);
                const uint32_t kt = (s.tile0 + t) * C::KT + key;  // this thread's key, its place
                const bool tail = (s.tile0 + t + 1) * C::KT > s.past;
                // bit per row: attended
                uint32_t on[RB / 32];
#pragma unroll
                for (int w = 0; w < RB / 32; ++w) on[w] = 0xffffffffu;
                uint32_t kp = kt;
                if (SC || tail) {
                    const bool in_tree = kt >= s.past;
                    const uint32_t j = kt - s.past;
                    const bool real = kt < s.past + s.n;
                    if (in_tree && real) kp = s.past + P.depth[s.s0 + j];
                    if (SC) {
                        if (P.rule.cap_out != 0.f) cap_scores<RB>(x, P.rule, series);
                        if (P.rule.slopes) {
#pragma unroll
                            for (int c = 0; c < RB; ++c)
                                x[c] = fmaf(-sloper[c], static_cast<float>(static_cast<int>(posr[c] - kp)), x[c]);
                        }
                    }
#pragma unroll
                    for (int w = 0; w < RB / 32; ++w) {
                        uint32_t m = 0;
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!SC || kp >= lor[32 * w + c]) m |= 1u << c;
                        if (in_tree) {
                            uint32_t in = 0;
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                const uint32_t row = 32 * w + c;
                                if (real && row < s.rows) {
                                    const uint32_t node = (s.row0 + row) / G;
                                    in |= (P.anc[static_cast<size_t>(s.s0 + node) * kTreeWords + j / 32] >>
                                           (j % 32) & 1u) << c;
                                }
                            }
                            m &= in;
                        }
                        on[w] = m;
                    }
                }
                // by how much the scores pass the maxima
                float over = -1e30f;
#pragma unroll
                for (int c = 0; c < RB; ++c)
                    if (on[c / 32] >> (c % 32) & 1u && c < static_cast<int>(Rp)) over = fmaxf(over, x[c] - ms[c]);
                const bool raise = bar_or(1, over > 8.f || !ok);
                bool wrote = false;
                if (raise) {
                    ok = !bar_or(1, !ok);
                    if (ok) {
                        // every row's maximum over the tile (as integers in the same order)
#pragma unroll
                        for (int c = 0; c < RB; ++c) {
                            const bool use = on[c / 32] >> (c % 32) & 1u && x[c] == x[c];
                            const int b = __float_as_int(use ? x[c] : -1e30f);
                            const int top = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
                            if (lane == 0) tmax[warp * RB + c] = __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
                        }
                        // P's buffer is free, so the accumulators have read the last factors
                        if (t != s.t0) ok = warp_wait(PE, (gt - 1) & 1);
                        wrote = true;
                        bar_128(1);
                        if (tid < RB) {
                            const float top = fmaxf(fmaxf(tmax[tid], tmax[RB + tid]),
                                                    fmaxf(tmax[2 * RB + tid], tmax[3 * RB + tid]));
                            const float old = ms[tid], m = fmaxf(old, top);
                            // (not 0: an infinity that the row holds has to stay one)
                            fs[tid] = fmaxf(tree_exp2(old - m), 1.17549435e-38f);
                            ms[tid] = m;
                        }
                        bar_128(1);
                    }
                }
#pragma unroll
                for (int c = 0; c < RB; ++c)
                    x[c] = on[c / 32] >> (c % 32) & 1u ? tree_exp2(x[c] - ms[c]) : -0.f;
                if (!wrote && t != s.t0) ok = warp_wait(PE, (gt - 1) & 1) && ok;
                // P^T: [32-key blocks][hi rows | lo rows][128 B]
                uint8_t* dst = smem + C::OFF_P + warp * (2 * Rp * 128) + (lane & 3) * 4;
#pragma unroll
                for (int c = 0; c < RB; ++c) {
                    if (c < static_cast<int>(Rp)) {
                        uint8_t* d = dst + c * 128 + (((lane >> 2) ^ (c & 7)) << 4);
                        *reinterpret_cast<float*>(d) = x[c];
                        *reinterpret_cast<float*>(d + Rp * 128) = x[c] - __uint_as_float(tf32_part(x[c]));
                    }
                }
                if (tid == 0) misc[1] = raise ? 1u : 0u;
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(PF);
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ converters
        const int w = warp - 4, me = w * 32 + lane;
        const uint32_t tlane = tb + (static_cast<uint32_t>(w) << 21);
        uint32_t pc = 0, kc = 0, vc = 0, gt = 0;  // pieces, K and V ones, tiles whose V is done
        auto k_tile = [&]() {
            for (int j = 0; j < C::KP; ++j, ++pc, ++kc) {
                const uint32_t sl = pc % NSLOT, b = kc % C::NKL;
                bool ok = warp_wait(FULL + 8 * sl, (pc / NSLOT) & 1);
                if (kc >= C::NKL) ok = warp_wait(KLE + 8 * b, (kc / C::NKL - 1) & 1) && ok;
                tc::fence_after_sync();
                const uint8_t* src = smem + C::OFF_RING + sl * C::PIECE + me * 128;
                uint32_t lo[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float4 x = *reinterpret_cast<const float4*>(src + ((c ^ (me & 7)) << 4));
                    lo[4 * c] = __float_as_uint(x.x - __uint_as_float(tf32_part(x.x)));
                    lo[4 * c + 1] = __float_as_uint(x.y - __uint_as_float(tf32_part(x.y)));
                    lo[4 * c + 2] = __float_as_uint(x.z - __uint_as_float(tf32_part(x.z)));
                    lo[4 * c + 3] = __float_as_uint(x.w - __uint_as_float(tf32_part(x.w)));
                }
                tc::tmem_st32(tlane + C::C_KL + 32 * b, lo);
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(KLF + 8 * b);
            }
        };
        auto v_tile = [&](uint32_t t) {
            // keys of the tile that the request has
            const uint32_t end = s.past + s.n - (s.tile0 + t) * C::KT;
            for (int j = 0; j < C::VP; ++j, ++pc, ++vc) {
                const uint32_t sl = pc % NSLOT, b = vc % C::NV;
                const uint32_t k0 = j / C::DH * C::VK;
                bool ok = warp_wait(FULL + 8 * sl, (pc / NSLOT) & 1);
                const int dim = me % C::VD;
                const float* src = reinterpret_cast<const float*>(smem + C::OFF_RING + sl * C::PIECE) + dim;
                uint32_t x[C::VK];
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < C::VK; ++k) {
                    x[k] = k0 + k < end ? __float_as_uint(src[k * C::VD]) : 0u;
                    top = max(top, x[k] & 0x7FFFFFFFu);
                }
                if (__any_sync(0xffffffffu, top >= 0x7F800000u)) {
#pragma unroll
                    for (int k = 0; k < C::VK; ++k)
                        if ((x[k] & 0x7F800000u) == 0x7F800000u) x[k] = 0u;
                    if (lane == 0) misc[2 + (gt & 1)] = gt + 1;
                }
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(VE + 8 * sl);
                if (vc >= C::NV) ok = warp_wait(VFE + 8 * b, (vc / C::NV - 1) & 1) && ok;
                tc::fence_after_sync();
                const uint32_t dst = tlane + C::C_V + C::VCOLS * b;
#pragma unroll
                for (int c = 0; c < C::VK / 32; ++c) {
                    uint32_t y[32];
                    if (C::FOLD) {
                        const bool low = w >= 2;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const uint32_t h = x[32 * c + k] & 0xFFFFE000u;
                            y[k] = low ? __float_as_uint(__uint_as_float(x[32 * c + k]) - __uint_as_float(h)) : h;
                        }
                        tc::tmem_st32(dst + 32 * c, y);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) y[k] = x[32 * c + k];
                        tc::tmem_st32(dst, y);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            y[k] = __float_as_uint(__uint_as_float(y[k]) - __uint_as_float(y[k] & 0xFFFFE000u));
                        tc::tmem_st32(dst + 32, y);
                    }
                }
                tc::tmem_st_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(VF + 8 * b);
            }
            ++gt;
        };
        while (walk.next(P, s)) {
            k_tile();
            for (uint32_t t = s.t0; t < s.t1; ++t) {
                if (t + 1 < s.t1) k_tile();
                v_tile(t);
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ accumulators
        grid_dependency_wait();
        const int w = warp - 8, me = w * 32 + lane;
        const uint32_t tlane = tb + (static_cast<uint32_t>(w) << 21);
        const float* ms = reinterpret_cast<const float*>(smem + C::OFF_M);
        const float* fs = reinterpret_cast<const float*>(smem + C::OFF_F);
        float* ls = reinterpret_cast<float*>(smem + C::OFF_L);
        constexpr int TPR = 128 / RB, KPT = C::KT / TPR;  // threads per row of P, keys of each
        const int lrow = me / TPR, lpart = me % TPR;
        bool ok = true;
        uint32_t gt = 0;
        while (walk.next(P, s)) {
            const uint32_t Rp = (s.rows + 15) / 16 * 16;
            float o[C::DH][RB];
#pragma unroll
            for (int d = 0; d < C::DH; ++d)
#pragma unroll
                for (int c = 0; c < RB; ++c) o[d][c] = 0.f;
            float l = 0.f;
            for (uint32_t t = s.t0; t < s.t1; ++t, ++gt) {
                ok = warp_wait(PF, gt & 1) && ok;
                if (misc[1]) {  // the maxima were raised: what there is shrinks
                    l *= fs[lrow];
#pragma unroll
                    for (int c = 0; c < RB; ++c) {
                        const float f = fs[c];
#pragma unroll
                        for (int d = 0; d < C::DH; ++d) o[d][c] *= f;
                    }
                }
                if (lrow < static_cast<int>(Rp)) {
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < KPT / 4; ++c) {
                        const int k = lpart * KPT + 4 * c;  // keys k .. k + 3
                        // (the two threads of a row read different banks)
                        const int q = (k / 4 & 7) ^ (lpart & 1) * 4;
                        const float4 p = *reinterpret_cast<const float4*>(
                            smem + C::OFF_P + k / 32 * (2 * Rp * 128) + lrow * 128 + ((q ^ (lrow & 7)) << 4));
                        sum[0] += p.x;
                        sum[1] += p.y;
                        sum[2] += p.z;
                        sum[3] += p.w;
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
                ok = warp_wait(OF, gt & 1) && ok;
                tc::fence_after_sync();
                const bool odd = misc[2 + (gt & 1)] == gt + 1;  // V values that are not finite
                if (!odd) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(PE);
                }
#pragma unroll
                for (int d = 0; d < C::DH; ++d) {
#pragma unroll
                    for (int c = 0; c < RB / 16; ++c) {
                        if (c * 16 >= static_cast<int>(Rp)) break;
                        uint32_t a[16], b[16];
                        tc::tmem_ld16(tlane + C::C_O + d * 2 * RB + 16 * c, a);
                        tc::tmem_ld16(tlane + C::C_O + d * 2 * RB + Rp + 16 * c, b);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            o[d][16 * c + k] += __uint_as_float(a[k]) + __uint_as_float(b[k]);
                    }
                }
                tc::fence_before_sync();
                if (odd) {
                    const uint32_t k0 = (s.tile0 + t) * C::KT;
                    const uint32_t end = min(s.past + s.n - k0, static_cast<uint32_t>(C::KT));
                    if (!C::FOLD || me < C::VD) {
                        for (uint32_t k = 0; k < end; ++k) {
                            const size_t place = tree_place(P, s.r, k0 + k);
#pragma unroll
                            for (int d = 0; d < C::DH; ++d) {
                                const float v = P.V[(place * P.n_kv_head + s.g) * HD + d * C::VD + me];
                                if ((__float_as_uint(v) & 0x7F800000u) != 0x7F800000u) continue;
#pragma unroll
                                for (int c = 0; c < RB; ++c) {
                                    if (c >= static_cast<int>(s.rows)) break;
                                    const uint32_t p = *reinterpret_cast<const uint32_t*>(
                                        smem + C::OFF_P + k / 32 * (2 * Rp * 128) + c * 128 +
                                        (((k / 4 & 7) ^ (c & 7)) << 4) + (k & 3) * 4);
                                    if (p != 0x80000000u) o[d][c] += v;
                                }
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(PE);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(OE);
            }
            // the unit's end: the rows' sums to everyone, then out or the partial
#pragma unroll
            for (int off = 1; off < TPR; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
            if (lpart == 0) ls[lrow] = l;
            const bool write = !bar_or(2, !ok);
            if (C::FOLD) {  // the products with V's low parts, through P's buffer
                float* fold = reinterpret_cast<float*>(smem + C::OFF_P);
                if (me >= 64) {
#pragma unroll
                    for (int c = 0; c < RB; ++c) fold[c * 64 + me - 64] = o[0][c];
                }
                bar_128(2);
                if (me < 64) {
#pragma unroll
                    for (int c = 0; c < RB; ++c) o[0][c] += fold[c * 64 + me];
                }
            }
            const bool whole = s.t0 == 0 && s.t1 == s.tl;
            if (write && P.req_of[s.s0] == s.r && (!C::FOLD || me < 64)) {
                const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (s.t0 == 0 ? 1 : 0);
                uint32_t node = s.row0 / G, h = s.row0 % G;
#pragma unroll
                for (int c = 0; c < RB; ++c) {
                    if (c >= static_cast<int>(s.rows)) break;
                    const float sum = ls[c], m = ms[c];
                    if (whole) {
                        float den = sum;
                        if (P.sinks) den += tree_exp2(__ldg(P.sinks + s.g * G + h) * kRuleLog2e - m);
                        const float inv = den == 0.f ? 0.f : 1.f / den;
                        float* dst = P.out + (static_cast<size_t>(s.s0 + node) * P.n_head + s.g * G + h) * HD + me;
#pragma unroll
                        for (int d = 0; d < C::DH; ++d) dst[d * C::VD] = o[d][c] * inv;
                    } else {
                        float* dst = P.part + (slot * RB + c) * HD + me;
#pragma unroll
                        for (int d = 0; d < C::DH; ++d) dst[d * C::VD] = o[d][c];
                        if (me == 0)
                            *reinterpret_cast<float2*>(P.part_ml + 2 * (slot * RB + c)) = make_float2(m, sum);
                    }
                    if (++h == G) {
                        h = 0;
                        ++node;
                    }
                }
            }
            bar_128(2);  // everyone has read the sums, the maxima and the fold's rows ...
            if (lane == 0) mbar_arrive(UE);  // ... which are the next unit's from here on
        }
    } else if (warp == 12) {
        // ------------------------------------------------------------ producer
        bool ok = true, waited = false;
        uint32_t pc = 0;
        uint32_t was_v = 0, ke = 0, ve = 0;  // per slot: its last piece was V; phases of its waits
        const uint32_t box = P.box_keys, boxes = C::KT / box;
        // the row of this lane's box in a tile
        auto rows_of = [&](uint32_t t) {
            const uint32_t k = (s.tile0 + t) * C::KT + lane * box;
            if (static_cast<uint32_t>(lane) >= boxes || k >= s.past + s.n) return 0u;
            return tree_place(P, s.r, k);
        };
        auto slot_free = [&](uint32_t sl) {
            if (pc < NSLOT) return;
            const uint32_t bit = 1u << sl;
            const bool v = was_v & bit;
            ok = warp_wait((v ? VE : KE) + 8 * sl, (v ? ve : ke) & bit ? 1 : 0) && ok;
            (v ? ve : ke) ^= bit;
        };
        auto k_tile = [&](uint32_t y) {
            for (int j = 0; j < C::KP; ++j, ++pc) {
                const uint32_t sl = pc % NSLOT;
                slot_free(sl);
                if (!ok) continue;
                was_v &= ~(1u << sl);
                if (lane == 0) mbar_expect_tx(FULL + 8 * sl, C::PIECE);
                __syncwarp();
                if (static_cast<uint32_t>(lane) < boxes)
                    tma_load_2d(sbase + C::OFF_RING + sl * C::PIECE + lane * box * 128, &tmK,
                                static_cast<int>(s.g * HD + 32 * j), static_cast<int>(y), FULL + 8 * sl);
            }
        };
        const uint32_t vbox = min(box, static_cast<uint32_t>(C::VK)), vboxes = C::VK / vbox;
        auto v_tile = [&](uint32_t y) {
            for (int j = 0; j < C::VP; ++j, ++pc) {
                const uint32_t sl = pc % NSLOT;
                slot_free(sl);
                const uint32_t k = j / C::DH * C::VK + lane * vbox;  // key of this lane's box
                const uint32_t row = __shfl_sync(0xffffffffu, y, (k / box) & 31) + k % box;
                if (!ok) continue;
                was_v |= 1u << sl;
                if (lane == 0) mbar_expect_tx(FULL + 8 * sl, C::PIECE);
                __syncwarp();
                if (static_cast<uint32_t>(lane) < vboxes)
                    tma_load_2d(sbase + C::OFF_RING + sl * C::PIECE + lane * vbox * C::VD * 4, &tmV,
                                static_cast<int>(s.g * HD + j % C::DH * C::VD), static_cast<int>(row),
                                FULL + 8 * sl);
            }
        };
        while (walk.next(P, s)) {
            // tiles of history may be read while the prep kernel still runs
            auto ready = [&](uint32_t t) {
                if (!waited && (s.tile0 + t + 1) * C::KT > s.past) {
                    grid_dependency_wait();
                    waited = true;
                }
            };
            ready(s.t0);
            uint32_t y = rows_of(s.t0);
            k_tile(y);
            for (uint32_t t = s.t0; t < s.t1; ++t) {
                uint32_t y1 = 0;
                if (t + 1 < s.t1) {
                    ready(t + 1);
                    y1 = rows_of(t + 1);
                    k_tile(y1);
                }
                v_tile(y);
                y = y1;
            }
        }
        grid_launch_dependents();
        if (misc[0])  // copies that may still be in flight
            for (uint32_t u = pc > NSLOT ? pc - NSLOT : 0; u < pc; ++u)
                mbar_wait(FULL + 8 * (u % NSLOT), (u / NSLOT) & 1, 1ll << 28);
    } else {
        // ------------------------------------------------------------ MMA issuer
        const bool lead = tc::elect_one();
        bool ok = true;
        uint32_t pc = 0, kc = 0, vc = 0, gs = 0, gp = 0, units = 0;  // pieces, tiles of S and of PV
        const uint64_t kdesc0 = tc::smem_desc(sbase + C::OFF_RING, 16, 1024, tc::kSwizzle128B);
        const uint64_t qdesc0 = tc::smem_desc(sbase, 16, 1024, tc::kSwizzle128B);
        const uint64_t pdesc0 = tc::smem_desc(sbase + C::OFF_P, 16, 1024, tc::kSwizzle128B);
        while (walk.next(P, s)) {
            const uint32_t Rp = (s.rows + 15) / 16 * 16;
            const uint32_t i2 = tc::idesc_tf32(128, 0, false) | (2 * Rp >> 3) << 17;
            const uint32_t i1 = tc::idesc_tf32(128, 0, false) | (Rp >> 3) << 17;
            const uint32_t block = 2 * Rp * 128 >> 4;  // a 32-wide block of Q or P
            ok = warp_wait(QF, units & 1) && ok;
            ++units;
            auto s_tile = [&]() {
                if (gs) ok = warp_wait(SE, (gs - 1) & 1) && ok;
                for (int j = 0; j < C::KP; ++j, ++pc, ++kc) {
                    const uint32_t sl = pc % NSLOT, b = kc % C::NKL;
                    ok = warp_wait(FULL + 8 * sl, (pc / NSLOT) & 1) && ok;
                    ok = warp_wait(KLF + 8 * b, (kc / C::NKL) & 1) && ok;
                    if (!ok) continue;
                    tc::fence_after_sync();
                    if (lead) {
                        const uint64_t kd = kdesc0 + (sl * C::PIECE >> 4), qd = qdesc0 + j * block;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            tc::mma_tf32_ss(tb + C::C_S, kd + 2 * kk, qd + 2 * kk, i2, j | kk ? 1u : 0u);
                            tc::mma_tf32_ts(tb + C::C_S + Rp, tb + C::C_KL + 32 * b + 8 * kk, qd + 2 * kk, i1, 1u);
                        }
                        tc::mma_commit(KE + 8 * sl);
                        tc::mma_commit(KLE + 8 * b);
                    }
                    __syncwarp();
                }
                // (the failure-path test option withholds the CTA's first score-ready signal)
                if (lead && ok && !(gs == 0 && (P.flags & kOptTestStall))) tc::mma_commit(SF);
                __syncwarp();
                ++gs;
            };
            s_tile();
            for (uint32_t t = s.t0; t < s.t1; ++t, ++gp) {
                if (t + 1 < s.t1) s_tile();
                ok = warp_wait(PF, gp & 1) && ok;
                if (gp) ok = warp_wait(OE, (gp - 1) & 1) && ok;
                for (int j = 0; j < C::VP; ++j, ++pc, ++vc) {
                    const uint32_t b = vc % C::NV;
                    ok = warp_wait(VF + 8 * b, (vc / C::NV) & 1) && ok;
                    if (!ok) continue;
                    tc::fence_after_sync();
                    if (lead) {
                        const uint32_t a = tb + C::C_V + C::VCOLS * b, d = tb + C::C_O + j % C::DH * 2 * RB;
                        const uint32_t k0 = j / C::DH * C::VK;
#pragma unroll
                        for (int kk = 0; kk < C::VK / 8; ++kk) {
                            const uint64_t pd = pdesc0 + (k0 + 8 * kk) / 32 * block + 2 * (kk % 4);
                            const uint32_t acc = j >= C::DH || kk ? 1u : 0u;
                            tc::mma_tf32_ts(d, a + 8 * kk, pd, i2, acc);
                            if (!C::FOLD) tc::mma_tf32_ts(d + Rp, a + 32 + 8 * kk, pd, i1, 1u);
                        }
                        tc::mma_commit(VFE + 8 * b);
                    }
                    __syncwarp();
                }
                if (lead && ok) {
                    tc::mma_commit(PE);
                    tc::mma_commit(OF);
                }
                __syncwarp();
            }
        }
        // every MMA has ended before tensor memory is freed
        if (lead) tc::mma_commit(DRAIN);
        __syncwarp();
        mbar_wait(DRAIN, 0);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 13) tc::tmem_dealloc(tb, C::TMEM_COLS);
}

// ------------------------------------------------------------------ combine
// One warp per (node, query head): the partial results of a unit that lies in
// several CTAs, in CTA order; the others are done already.
constexpr int kJoinThreads = 256;
template <int HD>
__global__ void __launch_bounds__(kJoinThreads) slotkv_tree_combine_kernel(const TreeParams P, uint32_t grid) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int RB = TreeCfg<HD>::RB, E = HD / 32;
    const int lane = threadIdx.x & 31;
    const uint64_t w = static_cast<uint64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const uint32_t tok = static_cast<uint32_t>(w / P.n_head), h = static_cast<uint32_t>(w % P.n_head);
    if (tok >= P.n_tok) return;
    const uint32_t r = P.req_of[tok];
    if (r >= P.n_req) return;
    const TreeShape x = tree_shape<RB>(P, r);
    if (x.nb == 0 || tok < x.q.s0 || tok - x.q.s0 >= x.q.n) return;  // (left from an earlier call)
    const uint32_t G = P.n_head / P.n_kv_head, g = h / G;
    const uint32_t row = (tok - x.q.s0) * G + h % G;
    const uint64_t total = P.base[P.n_req], a = P.base[r] + (static_cast<uint64_t>(g) * x.nb + row / RB) * x.tl;
    const uint32_t ctas = tree_ctas(total, grid);
    const uint32_t c0 = tree_owner(total, ctas, a), c1 = tree_owner(total, ctas, a + x.tl - 1);
    if (c0 == c1) return;
    auto slot = [&](uint32_t c) { return (2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0)) * RB + row % RB; };
    float m = -1e30f;
    for (uint32_t c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, __ldcg(P.part_ml + 2 * slot(c)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float den = 0.f, acc[E] = {};
    for (uint32_t c = c0; c <= c1; ++c) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(P.part_ml) + slot(c));
        const float f = fmaxf(tree_exp2(ml.x - m), 1.17549435e-38f);  // (see the raise)
        den = fmaf(ml.y, f, den);
        const float* src = P.part + slot(c) * HD + lane;
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] = fmaf(__ldcg(src + 32 * j), f, acc[j]);
    }
    if (P.sinks) den += tree_exp2(__ldg(P.sinks + h) * kRuleLog2e - m);
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int j = 0; j < E; ++j) P.out[(static_cast<size_t>(tok) * P.n_head + h) * HD + lane + 32 * j] = acc[j] * inv;
}

template <int HD>
int launch_tree_hd(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, uint32_t sms,
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
    const uint32_t groups = (p.n_head + kTreeQHeads - 1) / kTreeQHeads +
                            (p.n_kv_head + kTreeKvHeads - 1) / kTreeKvHeads;
    const uint64_t mean = (p.n_tok + p.n_req - 1) / p.n_req;
    const uint64_t parts = (mean * groups + kPrepWarps - 1) / kPrepWarps;
    cfg.gridDim = dim3(p.n_req, static_cast<unsigned>(parts < 256 ? parts : 256));
    cfg.blockDim = dim3(kPrepThreads);
    cfg.dynamicSmemBytes = tree_prep_smem<HD>();
    if ((e = cudaLaunchKernelEx(&cfg, slotkv_tree_prep_kernel<HD>, p)) != cudaSuccess) return static_cast<int>(e);
    cfg.gridDim = dim3(sms);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    const bool rule = p.rule.cap_out != 0.f || p.rule.window || p.rule.slopes || p.rule.doc_start;
    e = rule ? cudaLaunchKernelEx(&cfg, slotkv_tree_attn_kernel<HD, true>, tmK, tmV, p)
             : cudaLaunchKernelEx(&cfg, slotkv_tree_attn_kernel<HD, false>, tmK, tmV, p);
    if (e != cudaSuccess) return static_cast<int>(e);
    const uint64_t warps = static_cast<uint64_t>(p.n_tok) * p.n_head;
    cfg.gridDim = dim3(static_cast<unsigned>((warps + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, slotkv_tree_combine_kernel<HD>, p, sms));
}

}  // namespace slotkv
