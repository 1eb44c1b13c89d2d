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
#include "tree_attn.h"

namespace slotkv {

// Place p of request r in the [rows][kv_dim] view (p in range, its block in the pool).
__device__ __forceinline__ uint32_t tree_row(const TreeParams& P, uint32_t r, uint32_t p) {
    if (P.block_tables)
        return __ldg(P.block_tables + static_cast<size_t>(r) * P.bt_stride + p / P.slot_ctx) * P.slot_ctx +
               p % P.slot_ctx;
    return __ldg(P.slots + r) * P.slot_ctx + p;
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
// One warp per (node, query head): one pass over the keys with a running
// maximum and sum.
constexpr int kTreeThreads = 256;

template <int HD>
__global__ void __launch_bounds__(kTreeThreads) slotkv_tree_attn_kernel(const TreeParams P) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int E = HD / 32;
    const int lane = threadIdx.x & 31;
    const uint64_t w = static_cast<uint64_t>(blockIdx.x) * (kTreeThreads / 32) + (threadIdx.x >> 5);
    const uint32_t tok = static_cast<uint32_t>(w / P.n_head), h = static_cast<uint32_t>(w % P.n_head);
    if (tok >= P.n_tok) return;
    const uint32_t r = P.req_of[tok];
    if (r >= P.n_req) return;
    const TreeReq q = tree_request(P, r);
    if (!q.ok || tok < q.s0 || tok - q.s0 >= q.n) return;  // (left from an earlier call)
    const uint32_t pos = q.past + P.depth[tok], kvh = h / (P.n_head / P.n_kv_head);
    const uint32_t lo = rule_first(P.rule, r, pos);
    const float slope2 = P.rule.slopes ? P.rule.slopes[h] * kRuleLog2e : 0.f;
    float x[E], acc[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
        x[j] = P.q_rot[(static_cast<size_t>(tok) * P.n_head + h) * HD + lane + 32 * j];
        acc[j] = 0.f;
    }
    float m = -CUDART_INF_F, l = 0.f;
    for (uint32_t t = lo < q.past ? lo : q.past; t < q.past + q.n; ++t) {
        uint32_t kp = t;
        if (t >= q.past) {
            const uint32_t i = t - q.past;
            if (!(P.anc[static_cast<size_t>(tok) * kTreeWords + i / 32] >> (i % 32) & 1u)) continue;
            kp = q.past + P.depth[q.s0 + i];
            if (kp < lo) continue;
        }
        const size_t at = (static_cast<size_t>(tree_row(P, r, t)) * P.n_kv_head + kvh) * HD;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) s = fmaf(x[j], P.K[at + lane + 32 * j], s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s = apply_rule(s, P.rule.cap_in, P.rule.cap_out, slope2, P.rule.slopes != nullptr,
                       static_cast<int>(pos - kp));
        const float m2 = fmaxf(m, s), f = m2 == -CUDART_INF_F ? 1.f : exp2f(m - m2);
        const float p = s == -CUDART_INF_F ? 0.f : exp2f(s - m2);
        l = fmaf(l, f, p);
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] = fmaf(p, P.V[at + lane + 32 * j], acc[j] * f);
        m = m2;
    }
    if (P.sinks) {
        const float sk = P.sinks[h] * kRuleLog2e, m2 = fmaxf(m, sk);
        if (m2 != -CUDART_INF_F) {
            const float f = exp2f(m - m2);
            l = fmaf(l, f, exp2f(sk - m2));
#pragma unroll
            for (int j = 0; j < E; ++j) acc[j] *= f;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int j = 0; j < E; ++j) P.out[(static_cast<size_t>(tok) * P.n_head + h) * HD + lane + 32 * j] = acc[j] * inv;
}

template <int HD>
int launch_tree_hd(const TreeParams& p, cudaStream_t stream) {
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, slotkv_tree_prep_kernel<HD>, p);
    if (e != cudaSuccess) return static_cast<int>(e);
    const uint64_t warps = static_cast<uint64_t>(p.n_tok) * p.n_head;
    cfg.gridDim = dim3(static_cast<unsigned>((warps + kTreeThreads / 32 - 1) / (kTreeThreads / 32)));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = 0;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, slotkv_tree_attn_kernel<HD>, p));
}

}  // namespace slotkv
