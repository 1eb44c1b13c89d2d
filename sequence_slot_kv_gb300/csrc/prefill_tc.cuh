// prefill_tc.cuh -- batched causal prefill on the tensor cores, for head dims
// 64 and 128 ("Forward Cuda Gemma", prefillBatched: all prompt tokens of a
// call at once, equal to running them one decode step at a time; "Forward
// Cuda", batched prefill into the given slot).
//
// Three kernels per call, on one stream (the plan launched first, prep
// beside it as a programmatic dependent, the attention kernel after both):
//   * slotkv_prefill_prep_kernel: one warp per (token, 8 query heads or 4 kv
//     heads).  Query heads:
//     q' = RoPE(RMSnorm(q) * w) * scale * log2(e) into a workspace; kv heads:
//     k' = RoPE(RMSnorm(k_new) * w) and v into the token's slot row.  The
//     vector routines are the decode kernel's, so q' and k' are the same
//     bits as a decode step's.
//   * slotkv_prefill_plan_kernel (one CTA): cuts each run of consecutive
//     same-slot tokens into tiles of MT = 128 / G tokens -- a tile's G query
//     heads per token make the 128 rows of one MMA -- and lists the tiles,
//     handed out in reverse (each run from its last tile to its first).  A
//     work item is one (tile, kv head): keys 0 .. the tile's largest
//     position, read once for all its rows.
//   * slotkv_prefill_tc_kernel (persistent, one CTA per SM): flash attention
//     of each item with f32 accuracy from TF32 tensor-core products, split
//     in three: a = a_hi + a_lo with a_hi = a with its low 13 mantissa bits
//     cleared (exact in TF32) and a_lo = a - a_hi (exact in f32), and
//     a.b ~ a_hi.b_hi + a_hi.b_lo + a_lo.b_hi (the dropped a_lo.b_lo and the
//     TF32 rounding of the lo parts are ~2^-20 relative).
//       - warp 8 (producer): claims items and streams each key tile's K
//         and then V (BK = 64 keys x hd, 128-byte swizzled boxes of 32
//         floats) with TMA into a ring of half-stage slots (one operand's
//         hi and lo buffers each: 3 slots for hd 128, 6 for hd 64 and for
//         scored calls);
//       - warps 10-13 (converters): write each landed K tile's lo part
//         beside it (the tensor core reads a TF32 operand's f32 bits with the
//         low 13 mantissa bits ignored, so the landed tile is its own hi
//         part), and transpose each landed V tile into
//         a keys-contiguous layout while splitting it (TF32 MMA operands
//         in shared memory are K-major: for O += P V that is V^T, [hd][keys]);
//         keys past the item's last are zeroed;
//       - warp 9 (MMA issuer, one thread): S = Q K^T into a TMEM score
//         buffer (A = Q from TMEM), then O += P V (A = P from TMEM, B = the
//         transposed V tile).  With two score buffers (hd 64) the issue order
//         is QK(t+1), PV(t), QK(t+2), ...; with one (hd 128, where Q's hi and
//         lo parts take half of tensor memory) QK(t), PV(t), QK(t+1), ....
//         MMAs from one thread run in issue order, so a QK reuses a buffer
//         only after the PV before it has read it;
//       - warps 0-7 (softmax; two threads per query row = TMEM lane, each
//         with half of the columns, combining maxima and sums at pairwise
//         named barriers): put the item's q rows (hi, lo) into TMEM -- the
//         next item's as soon as the current item's last P is written, so
//         the next item's first QK overlaps the current item's epilogue --
//         then per key tile read S,
//         apply the causal mask (key <= the row's position), run a base-2
//         online softmax with a lazily raised max, write P (hi over S, lo
//         beside it) into the same buffer and, only when the max moves,
//         wait for the previous PV and rescale O in TMEM; at the end read O,
//         normalise (sink included) and store out.
// Every mbarrier wait is bounded; on expiry the CTA raises SLOTKV_DEV_TIMEOUT
// and every role leaves its loop; the MMA thread waits for its MMAs and the
// producer for its copies before tensor memory is freed.  The test option
// SLOTKV_OPT_TEST_STALL withholds each CTA's first score-ready signal to
// exercise that path.
//
// Scored calls (template parameter SC; parameters ScoredPrefillParams) are
// the same three kernels with the score rule of score_rule.cuh, and also the
// prefix pass of a shared decode call, whose rows attend the first
// prefix_lens[b] keys of another handle's slot.  What differs:
//   * each row has a key range [lo, hi]; a tile reads the union of its rows'
//     ranges, and scores outside a row's own range are masked;
//   * a call with few tiles cuts each tile's keys into splits (the plan picks
//     the chunk, see below): an item is then (tile, split, kv head), and it
//     leaves (m, l, O) in the partials instead of out.  The splits of a
//     prefill are joined by slotkv_combine_kernel, those of a prefix pass by
//     the decode kernel;
//   * sums that stay at f32 accuracy however many keys there are: the tensor
//     core's accumulation drops bits at every step, always toward zero, so a
//     long chain drifts (1.2e-4 relative over 16 thousand keys).  Each key
//     tile's P V therefore starts a new accumulator, which the softmax warps
//     add to a register copy of O with rounded f32 adds, and within a chain
//     the products with a low part come first, while the partial sum is still
//     small.  Q and P are split with a rounded high part, so the dropped
//     lo x lo terms have no common sign;
//   * two score buffers at head dim 128 too: its key tiles are 32 keys, not 64,
//     so Q, O and two buffers of (S, P) fill the 512 columns of tensor memory.
//     O has one buffer there: O(t - 1) is read once the softmax of tile t is
//     done, just before P(t) allows the tensor core to write O again.  At head
//     dim 64 O has two, and O(t - 2) is read with S(t);
//   * 16 warps: converters 10-13 take V and 14-15 K, so K(t + 1) and V(t) are
//     converted side by side; the MMA warp issues in step, one elected lane;
//     q and out rows pass through 2 KB of shared memory per softmax warp, in
//     64-byte pieces; the softmax's halves exchange maxima only when a row's
//     would rise;
//   * a V value that is not finite is taken as 0 by the tensor core (0 times
//     it would poison every masked row of the tile), and rows that do attend
//     it get it added in the epilogue from the slot itself.  The converters
//     keep a log of the key tiles that held one, so that only those are read
//     again, and only for the item they belong to: of 39 tiles of 16 tokens on
//     12000 keys, one infinity in another sequence of the call leaves the time
//     as it is (1.01 ms at head dim 64, 1.28 at 128), one in every 997th key
//     adds 0.1 to 0.2 ms; a history of nothing else takes 0.5 to 0.7 us a key.
//     The log costs the calls without any 0.6 to 1.3 %.
// Where they hold fewer bits than f32: the low parts of Q, K, V and P are cut
// to TF32 by the tensor core and the product of two low parts is left out.  K
// and V are split by truncation (K's landed tile is then its own high part, and
// is not written again), so their low parts reach 2^-10 of the value and each
// of the two losses 2^-20 of a product; the tests' bounds count those.
// Exponentials are ex2.approx.ftz and the cap divides by __fdividef, both a few
// ulp.  Against 64 bits the listed cases are off by 4e-7 to 7e-7 of the largest
// value, plain f32 forms by 2e-7 to 3e-6.
// What bounds them, measured: head dim 128, 256 rows on a prefix of 32700 keys,
// 502 us, 2120 cycles per tile of 32 keys of which the tensor core needs 1800
// (three TF32 products: 85 % of its rate); head dim 64, 517 tokens on 15.8
// thousand keys, 568 us, 2370 cycles per tile of 64 keys against 1800, the
// rest the softmax's latencies.  64-key tiles with one score buffer at head
// dim 128 took 636 us, a single thread issuing 33 % longer.
#pragma once

#include "decode_attn.cuh"
#include "tc_ops.cuh"

namespace slotkv {

template <int HD, int G, bool SC = false>
struct PCfg {
    static constexpr int M = 128;               // query rows per tile (MMA M)
    static constexpr int MT = M / G;            // tokens per tile
    static constexpr int ROWS = MT * G;         // rows in use (<= 128)
    static constexpr int BK = prefill_tile_keys(HD, SC);  // keys per tile (QK's N)
    static constexpr int NB = HD / 32;          // 128-byte column blocks per key row
    static constexpr int BLK = BK * 128;        // one column block: BK rows x 128 B
    static constexpr int BUF = NB * BLK;        // one operand buffer, [BK][HD] f32
    static constexpr int SLOT = 2 * BUF;        // half-stage slot: hi | lo of K or V
    static constexpr int NSLOT = (192 * 1024) / SLOT;  // 6; plain calls at hd 128: 3
    // V transposed: KB column blocks of 32 keys, each [HD rows][128 B]; the
    // 32 x 32 sub-block (key block kb, dim block db) lands at kb * VT_BLK +
    // db * 4096 (TMA put it at db * BLK + kb * 4096)
    static constexpr int KB = BK / 32;
    static constexpr int VT_BLK = HD * 128;
    // softmax warps: two per tensor-memory lane quarter (warps q and q + 4),
    // each taking half of a score tile's columns
    static constexpr int NSW = 8;
    static constexpr int WARP_TMA = 8, WARP_MMA = 9, WARP_CONV = 10, NCONV = 4;
    static constexpr int SB_PER_WARP = KB * NB / NCONV;  // V sub-blocks per converter warp
    static constexpr int THREADS = 32 * (WARP_CONV + NCONV);
    // scored calls: two more warps convert K while the four take V, so K(t + 1)
    // and V(t) are converted side by side; that makes whole warpgroups,
    // launched at 128 registers a thread, of which the two softmax ones, with O
    // in registers, take from the other two: 256 * 160 + 256 * 96 = 512 * 128
    static constexpr int NKCONV = 2;
    static constexpr int THREADS_SC = 512, REG_SOFTMAX = 160, REG_OTHER = 96;
    static_assert(256 * REG_SOFTMAX + 256 * REG_OTHER == THREADS_SC * 128,
                  "register hand-over must add up to the launch's registers");
    // tensor memory columns: Q hi | Q lo | O | NBUF buffers of (S, then P hi
    // over it | P lo)
    static constexpr uint32_t C_QHI = 0, C_QLO = HD, C_O = 2 * HD, C_S = 3 * HD;
    static constexpr uint32_t C_BUF = 2 * BK;   // columns per score buffer
    static constexpr int NBUF = (512 - 3 * HD) / (2 * BK) >= 2 ? 2 : 1;
    // scored calls: a second O after the score buffers where there is room
    // (head dim 64): O(t - 2) is then read together with S(t); with one, O(t -
    // 1) is read before P(t) is handed over (604 instead of 584 us for 517
    // tokens on 15.8 thousand keys)
    static constexpr uint32_t C_O2 = 3 * HD + NBUF * 2 * BK;
    static constexpr bool TWO_O = SC && NBUF == 2 && C_O2 + HD <= 512;
    static_assert(!SC || NBUF == 2, "scored calls: two score buffers");
    static constexpr uint32_t TMEM_COLS = 512;
    static_assert(3 * HD + NBUF * 2 * BK <= 512, "tensor memory columns");
    static_assert(BK % 32 == 0 && HD % 32 == 0, "32-column tensor memory accesses");
    // shared memory after the ring: item descriptors [2][8] | slot meta
    // [NSLOT][4] | barriers | tensor memory address | flags
    static constexpr int OFF_DESC = NSLOT * SLOT;
    static constexpr int OFF_META = OFF_DESC + 2 * 32;
    static constexpr int OFF_BAR = OFF_META + NSLOT * 16;
    // full[NSLOT], conv[NSLOT], empty[NSLOT], s_full[2], p_ready[2],
    // pv_done[2], q_ready, item_full[2], item_free[2], drain
    static constexpr int NBAR = 3 * NSLOT + 12;
    // (scored calls' converters see one kind of half-tile each: with an even
    // number of slots a slot, and its barriers, is always K's or always V's,
    // and they see every phase of theirs)
    static_assert(!SC || NSLOT % 2 == 0, "a slot is of one kind");
    static constexpr int OFF_TSLOT = OFF_BAR + NBAR * 8;
    static constexpr int OFF_MISC = OFF_TSLOT + 16;
    // misc[0]: abort; misc[2 + w]: converter warp w's stop flag
    // the softmax halves' exchange: row maxima [2 parities][2 halves][M],
    // row sums [2 halves][M], and a stop flag beside each
    static constexpr int OFF_XCH = OFF_MISC + 64;
    static constexpr int SMEM_USED = OFF_XCH + 2 * 6 * M * 4;
    static constexpr int SMEM = SMEM_USED + 1024;   // slack to align the ring to 1 KiB
    // scored calls: 2 KB for each softmax warp to stage rows in
    static constexpr int OFF_STAGE = (SMEM_USED + 15) / 16 * 16;
    // and each converter warp's log of the key tiles, numbered over the CTA's
    // items, that held a V value that is not finite: [NCONV][LOG] runs of
    // tiles (first, last), then the runs so far and the last tile plus 1
    static constexpr int LOG = 64, LOG_GAP = 8;
    static constexpr int OFF_LOG = OFF_STAGE + NSW * 2048;
    static constexpr int SMEM_SC = OFF_LOG + NCONV * (2 * LOG + 2) * 4 + 1024;
    static_assert(SMEM <= 227 * 1024 && SMEM_SC <= 227 * 1024, "shared memory");
    static_assert(BLK % 1024 == 0 && SLOT % 1024 == 0, "128-byte swizzle atoms stay 1 KiB aligned");
    static constexpr uint32_t IDESC_QK = tc::idesc_tf32(M, BK, false);
    static constexpr uint32_t IDESC_PV = tc::idesc_tf32(M, HD, false);
    static_assert(KB * NB == SB_PER_WARP * NCONV, "V sub-blocks split evenly over the converters");
};

// Named barrier 2 over the converter warps (N threads).
template <int N>
__device__ __forceinline__ void named_sync_conv() {
    asm volatile("bar.sync 2, %0;" ::"n"(N) : "memory");
}

// 2^x by the hardware's approximate base-2 exponential (PTX ex2.approx.ftz:
// a few ulp of relative error, subnormal results flushed to zero), far
// inside the f32 tolerance of the step.
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Split x into an exactly-TF32 high part and the f32 remainder.
__device__ __forceinline__ void tf32_split(float x, uint32_t& hi, uint32_t& lo) {
    const uint32_t h = __float_as_uint(x) & 0xFFFFE000u;
    hi = h;
    lo = __float_as_uint(x - __uint_as_float(h));
}

// The same for two values, with the high parts rounded to nearest, so a
// remainder is at most half a TF32 step and takes either sign (one packed
// subtraction).
__device__ __forceinline__ void tf32_split_rn2(float x, float y, uint32_t& hx, uint32_t& hy,
                                               uint32_t& lx, uint32_t& ly) {
    hx = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    hy = (__float_as_uint(y) + 0x1000u) & 0xFFFFE000u;
    const float2 d = __ffma2_rn(make_float2(__uint_as_float(hx), __uint_as_float(hy)),
                                make_float2(-1.f, -1.f), make_float2(x, y));
    lx = __float_as_uint(d.x);
    ly = __float_as_uint(d.y);
}

// ------------------------------------------------------------------ prep
// One warp per (token, group of heads): kPrepHeads query heads, or
// kPrepKvHeads kv heads (their k_new and v_new rows), so that every warp
// stages kPrepHeads rows.  The group's rows are staged into the warp's
// shared memory with cp.async, all in flight at once, while the warp forms
// the token's RoPE angles; then each row goes through the decode kernel's
// vector routine (the same arithmetic on the same values, so the same bits
// as a decode step).
constexpr int kPrepHeads = 8, kPrepKvHeads = kPrepHeads / 2;

__device__ __forceinline__ void prep_cp_async16(void* smem_dst, const void* gmem_src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem_dst)),
                 "l"(gmem_src)
                 : "memory");
}

// Row i of a scored call as the tensor-core kernels see it: the slot it reads
// (its own, or its prefix's), its key range there, its position; ok: in
// range; keys: it has keys in that slot for the tensor cores to attend (a
// prefill row always belongs to a tile, be its mask empty).
struct PrefillRow {
    uint32_t slot, pos, lo, hi;
    bool ok, keys;
};
__device__ __forceinline__ PrefillRow prefill_row(const ScoredPrefillParams& P, uint32_t i) {
    PrefillRow r;
    r.pos = __ldg(P.positions + i);
    r.slot = __ldg(P.slots + i);
    r.lo = rule_first(P.rule, i, r.pos);
    if (P.shared.lens) {
        const uint32_t own = __ldg(P.own_slots + i);
        const ScoredRow x = scored_row(P.rule, P.shared, i, r.pos, P.own_ctx,
                                       own < P.own_n_slots, false);
        r.ok = x.ok;
        r.keys = x.ok && x.len != 0u && r.lo < x.len;
        r.hi = r.keys ? x.len - 1u : 0u;
    } else {
        const ScoredRow x = scored_row(P.rule, P.shared, i, r.pos, P.slot_ctx,
                                       r.slot < P.n_slots, true);
        r.ok = r.keys = x.ok;
        r.hi = x.hi;
    }
    return r;
}

template <int HD>
__host__ __device__ constexpr int prep_smem_bytes(int warps = 4) {
    return warps * kPrepHeads * HD * 4;  // kPrepHeads rows per warp
}

// query-head groups and kv-head groups per token
__host__ __device__ inline uint32_t prep_q_groups(uint32_t n_head) {
    return (n_head + kPrepHeads - 1) / kPrepHeads;
}
__host__ __device__ inline uint32_t prep_groups(uint32_t n_head, uint32_t n_kv_head) {
    return prep_q_groups(n_head) + (n_kv_head + kPrepKvHeads - 1) / kPrepKvHeads;
}

// wg: the warp's place in the grid
template <int HD, bool SC>
__device__ __forceinline__ void prefill_prep(const prefill_params_t<SC>& P, const uint32_t wg) {
    extern __shared__ __align__(16) uint8_t prep_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t qg = prep_q_groups(P.n_head);
    uint32_t groups = prep_groups(P.n_head, P.n_kv_head);
    if constexpr (SC)
        if (P.shared.lens) groups = qg;  // the decode kernel forms and writes k' and v
    const uint32_t tok = wg / groups, grp = wg % groups;
    if (tok >= P.n_tok) return;
    const uint32_t p = P.positions[tok], slot = P.slots[tok];
    if constexpr (SC) {
        if (!prefill_row(P, tok).ok) return;
    } else {
        if (slot >= P.n_slots || p >= P.slot_ctx) return;  // the plan raises the flag
    }
    const bool is_q = grp < qg;
    // the group's first head (a query head, or a kv head) and its size
    const uint32_t x0 = is_q ? grp * kPrepHeads : (grp - qg) * kPrepKvHeads;
    const uint32_t left = (is_q ? P.n_head : P.n_kv_head) - x0;
    const uint32_t cap = is_q ? kPrepHeads : kPrepKvHeads;
    const uint32_t nx = left < cap ? left : cap;
    float* rows = reinterpret_cast<float*>(prep_smem) + warp * kPrepHeads * HD;
    float* vrows = rows + kPrepKvHeads * HD;  // kv groups: v rows after the k rows
    for (uint32_t i = 0; i < nx; ++i) {
        const uint32_t x = x0 + i;
        if (is_q) {
            const float* src = P.q + (static_cast<size_t>(tok) * P.n_head + x) * HD;
            for (int c = lane; c < HD / 4; c += 32) prep_cp_async16(rows + i * HD + 4 * c, src + 4 * c);
        } else {
            const size_t at = (static_cast<size_t>(tok) * P.n_kv_head + x) * HD;
            for (int c = lane; c < HD / 4; c += 32) {
                prep_cp_async16(rows + i * HD + 4 * c, P.k_new + at + 4 * c);
                prep_cp_async16(vrows + i * HD + 4 * c, P.v_new + at + 4 * c);
            }
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    float cs[HD / 64], sn[HD / 64];
    warp_rope_angles<HD>(p, P.inv_freq, cs, sn, lane);
    const float w1 = (P.flags & kOptNormPlusOne) ? 1.0f : 0.0f;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    for (uint32_t i = 0; i < nx; ++i) {
        const uint32_t x = x0 + i;
        if (is_q) {
            const size_t at = (static_cast<size_t>(tok) * P.n_head + x) * HD;
            warp_norm_rope<HD>(rows + i * HD, P.q_rot + at, P.q_norm_w, w1, P.scale_log2, P.eps,
                               cs, sn, lane);
            continue;
        }
        const size_t dst = ((static_cast<size_t>(slot) * P.slot_ctx + p) * P.n_kv_head + x) * HD;
        warp_norm_rope<HD>(rows + i * HD, P.K + dst, P.k_norm_w, w1, 1.0f, P.eps, cs, sn, lane);
        if (P.flags & kOptVNorm) {
            warp_rms_norm_plain<HD>(vrows + i * HD, P.V + dst, P.eps, lane);
        } else {
#pragma unroll
            for (int j = 0; j < HD / 32; ++j) P.V[dst + lane + 32 * j] = vrows[i * HD + lane + 32 * j];
        }
    }
}

template <int HD, bool SC = false>
__global__ void __launch_bounds__(128)
    slotkv_prefill_prep_kernel(const prefill_params_t<SC> P) {
    // scored calls: the attention kernel may be set up beside this one's end,
    // and the last CTA ends after the plan, this kernel's programmatic
    // predecessor
    if constexpr (SC) grid_launch_dependents();
    prefill_prep<HD, SC>(P, blockIdx.x * 4 + (threadIdx.x >> 5));
    if constexpr (SC)
        if (blockIdx.x == gridDim.x - 1) grid_dependency_wait();
}

// ------------------------------------------------------------------ plan
// One CTA of 1024 threads, tokens in rounds of 1024.  A run is a maximal
// sequence of consecutive in-range tokens with the same slot; token i starts
// a tile when its index within its run is a multiple of MT.  Tile records:
// (first token, tokens, slot, largest position).  Out-of-range tokens raise
// SLOTKV_DEV_RANGE and belong to no tile.  Then the tiles' hand-out order.

template <int MT>
__global__ void __launch_bounds__(1024, 1) slotkv_prefill_plan_kernel(const PrefillParams P) {
    __shared__ int warp_max[32];
    __shared__ uint32_t warp_sum[32];
    __shared__ int carry_start;
    __shared__ uint32_t carry_tiles;
    // The prep kernel, launched next as a programmatic dependent, may start
    // at once: it reads none of what this kernel writes and writes none of
    // what it reads, and the attention kernel after both waits for both.
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        carry_start = -1;
        carry_tiles = 0;
    }
    __syncthreads();
    uint4* tiles = reinterpret_cast<uint4*>(P.tiles);
    for (uint32_t r0 = 0; r0 < P.n_tok; r0 += 1024) {
        const uint32_t i = r0 + tid;
        bool valid = false, start = false;
        uint32_t slot = 0;
        if (i < P.n_tok) {
            slot = P.slots[i];
            valid = slot < P.n_slots && P.positions[i] < P.slot_ctx;
            if (!valid) atomicOr(P.status, kDevRange);
            if (valid) {
                if (i == 0) {
                    start = true;
                } else {
                    const uint32_t ps = P.slots[i - 1];
                    start = ps != slot || P.positions[i - 1] >= P.slot_ctx;
                }
            }
        }
        // the latest run start at or before i: an inclusive prefix max
        int a = start ? static_cast<int>(i) : -1;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, a, off);
            if (lane >= off) a = a > o ? a : o;
        }
        if (lane == 31) warp_max[warp] = a;
        __syncthreads();
        if (warp == 0) {
            int v = warp_max[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, v, off);
                if (lane >= off) v = v > o ? v : o;
            }
            warp_max[lane] = v;
        }
        __syncthreads();
        int rs = warp > 0 ? warp_max[warp - 1] : -1;
        rs = rs > carry_start ? rs : carry_start;
        rs = rs > a ? rs : a;
        const bool tflag = valid && ((i - static_cast<uint32_t>(rs)) % MT) == 0;
        // tile index: an inclusive prefix sum of the tile starts
        uint32_t c = tflag ? 1u : 0u;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, c, off);
            if (lane >= off) c += o;
        }
        if (lane == 31) warp_sum[warp] = c;
        __syncthreads();
        if (warp == 0) {
            uint32_t v = warp_sum[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, v, off);
                if (lane >= off) v += o;
            }
            warp_sum[lane] = v;
        }
        __syncthreads();
        const uint32_t incl = c + (warp > 0 ? warp_sum[warp - 1] : 0u) + carry_tiles;
        if (tflag) tiles[incl - 1] = make_uint4(i, 0u, slot, 0u);
        if (i < P.n_tok) P.tile_of[i] = valid ? incl - 1 : 0xFFFFFFFFu;
        __syncthreads();  // every thread has read the carries
        if (tid == 1023) {
            carry_start = rs;
            carry_tiles = incl;
        }
        __syncthreads();
    }
    // each tile's token count and largest position
    for (uint32_t i = tid; i < P.n_tok; i += 1024) {
        const uint32_t t = P.tile_of[i];
        if (t == 0xFFFFFFFFu) continue;
        uint32_t* rec = P.tiles + 4 * static_cast<size_t>(t);
        atomicAdd(rec + 1, 1u);
        atomicMax(rec + 3, P.positions[i]);
    }
    __syncthreads();
    // The hand-out order, into tile_of (its per-token use is over): the
    // tiles in reverse, so each run is handed out from its last tile (the
    // most keys, when its positions increase) to its first, one run after
    // the other -- the attention kernel ends on small items while a run's
    // keys stay in L2 across its tiles.  (Any order gives the same bits:
    // items are independent.)
    const uint32_t n_tiles = carry_tiles;
    for (uint32_t t = tid; t < n_tiles; t += 1024) P.tile_of[t] = n_tiles - 1 - t;
    __syncthreads();
    if (tid == 0) {
        P.plan[0] = carry_tiles * P.n_kv_head;
        P.plan[1] = 0;
    }
}

// The scored calls' plan (one CTA of NT threads, PER consecutive tokens per
// thread and round: 256 threads and one token for a call of up to 256 rows,
// 1024 and one up to 1024 -- the time of such a call is the latency of code run
// once, so the least of it and few warps to wait for: 4.3 us for six rows, 7.4
// for 517 -- else 1024 and eight).  Runs and tiles as above, over the rows that
// have keys for the tensor cores (PrefillRow); a tile's record is the same,
// with its smallest key in tile_lo.  The first kPlanTiles tiles are kept in
// shared memory until the end.
//
// With few tiles their keys are cut into splits, which fills the GPU and
// evens its items out: one chunk length for every tile, of the lengths that
// cut the longest tile into 1 .. kMaxSplits splits the one with the least
// estimated time -- waves of items over the SMs, times key tiles per item plus
// kItemCost for its q load, its epilogue and the join of its partial.  Items
// are listed split by split, so CTAs that run together share a split's keys
// in L2; unsplit tiles are listed last to first, as above.  The order has no
// part in any result: a split's partial has a place of its own.
constexpr uint32_t kPlanTiles = 512;
constexpr uint32_t kItemCost = 128, kMinChunk = 128;  // in keys

// Inclusive scan of one value per thread over the CTA.
template <typename T, typename Op>
__device__ T block_inclusive(T v, T* warp_vals, Op op, T zero) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v = op(v, o);
    }
    if (lane == 31) warp_vals[warp] = v;
    __syncthreads();
    T w = lane < warp ? warp_vals[lane] : zero;  // the warps before this one
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) w = op(w, __shfl_xor_sync(0xffffffffu, w, off));
    return op(v, w);
}

template <int MT, int BK, uint32_t NT, uint32_t PER>
__device__ __forceinline__ void scored_plan(const ScoredPrefillParams& P) {
    __shared__ uint32_t t_first[kPlanTiles], t_rows[kPlanTiles], t_slot[kPlanTiles];
    __shared__ uint32_t t_lo[kPlanTiles], t_hi[kPlanTiles], t_ns[kPlanTiles], t_part[kPlanTiles];
    __shared__ int scan_i[32];
    __shared__ uint32_t scan_u[32], hist[kMaxSplits + 1], at[kMaxSplits + 1];
    __shared__ uint32_t carry_tiles, longest;
    __shared__ int carry_start;
    __shared__ uint64_t best[kMaxSplits / 32];
    // the last token of the previous round and of each warp: its slot, and
    // whether it has keys
    __shared__ uint32_t last_of_slot[NT / 32 + 1], last_of_keys[NT / 32 + 1];
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint4* tiles = reinterpret_cast<uint4*>(P.tiles);
    uint4* rec = reinterpret_cast<uint4*>(P.part.rec);
    if (tid == 0) {
        carry_tiles = 0;
        carry_start = -1;
        longest = 1;
        last_of_keys[0] = 0;
    }
    if (tid <= kMaxSplits) hist[tid] = at[tid] = 0;
    __syncthreads();
    uint32_t own_tile = 0xFFFFFFFFu;  // of the thread's last token
    auto max_op = [](int a, int b) { return a > b ? a : b; };
    auto add_op = [](uint32_t a, uint32_t b) { return a + b; };
    for (uint32_t r0 = 0; r0 < P.n_tok; r0 += NT * PER) {
        const uint32_t i0 = r0 + tid * PER;
        uint32_t slot[PER], lo[PER], hi[PER];
        uint32_t keys = 0, starts = 0;  // bit j: token i0 + j
        uint32_t last_slot = 0, last_keys = 0;  // of the thread's last token
#pragma unroll
        for (uint32_t j = 0; j < PER; ++j) {
            slot[j] = lo[j] = hi[j] = 0;
            if (i0 + j < P.n_tok) {
                const PrefillRow r = prefill_row(P, i0 + j);
                if (!r.ok) atomicOr(P.status, kDevRange);
                keys |= (r.keys ? 1u : 0u) << j;
                rec[2 * (i0 + j) + 1] = make_uint4(r.pos, r.lo, r.hi, 0u);
                slot[j] = r.slot;
                hi[j] = r.hi;
                lo[j] = r.lo < r.hi ? r.lo : r.hi;
                last_slot = r.slot;
                last_keys = r.keys ? 1u : 0u;
            }
        }
        uint32_t prev_slot = __shfl_up_sync(0xffffffffu, last_slot, 1);
        uint32_t prev = __shfl_up_sync(0xffffffffu, last_keys, 1);
        if (lane == 31) {
            last_of_slot[warp + 1] = last_slot;
            last_of_keys[warp + 1] = last_keys;
        }
        __syncthreads();
        if (lane == 0) {
            prev_slot = last_of_slot[warp];
            prev = last_of_keys[warp];
        }
        int last_start = -1;
#pragma unroll
        for (uint32_t j = 0; j < PER; ++j) {
            if (keys >> j & 1u) {
                const bool follows = j ? (keys >> (j - 1) & 1u) && slot[j - 1] == slot[j]
                                       : prev && prev_slot == slot[j];
                if (!follows) {
                    starts |= 1u << j;
                    last_start = static_cast<int>(i0 + j);
                }
            }
        }
        // the run start before this thread's tokens, then its tile starts
        const int incl_start = block_inclusive(last_start, scan_i, max_op, -1);
        int before = __shfl_up_sync(0xffffffffu, incl_start, 1);
        if (lane == 0) {
            before = carry_start;
            for (uint32_t w = 0; w < warp; ++w) before = max_op(before, scan_i[w]);
        }
        before = max_op(before, carry_start);
        uint32_t opens = 0;
        int run = before;
#pragma unroll
        for (uint32_t j = 0; j < PER; ++j) {
            if (starts >> j & 1u) run = static_cast<int>(i0 + j);
            if ((keys >> j & 1u) && (i0 + j - static_cast<uint32_t>(run)) % MT == 0) opens |= 1u << j;
        }
        const uint32_t incl = block_inclusive(static_cast<uint32_t>(__popc(opens)), scan_u, add_op, 0u);
        uint32_t t = carry_tiles + incl - __popc(opens);  // tiles opened before
#pragma unroll
        for (uint32_t j = 0; j < PER; ++j) {
            if (opens >> j & 1u) {
                if (t < kPlanTiles) {
                    t_first[t] = i0 + j;
                    t_slot[t] = slot[j];
                    t_rows[t] = 0;
                    t_lo[t] = 0xFFFFFFFFu;
                    t_hi[t] = 0;
                } else {
                    tiles[t] = make_uint4(i0 + j, 0u, slot[j], 0u);
                    P.tile_lo[t] = 0xFFFFFFFFu;
                }
                ++t;
            }
        }
        __syncthreads();
        // each tile's rows, smallest and largest key: this thread's tokens
        // tile by tile; when one tile takes the whole warp, once for all
        t = carry_tiles + incl - __popc(opens);
        uint32_t n = 0, tlo = 0xFFFFFFFFu, thi = 0;
        auto flush = [&](uint32_t tile) {
            if (n == 0) return;
            uint32_t* rows = tile < kPlanTiles ? t_rows + tile : P.tiles + 4 * static_cast<size_t>(tile) + 1;
            uint32_t* plo = tile < kPlanTiles ? t_lo + tile : P.tile_lo + tile;
            uint32_t* phi = tile < kPlanTiles ? t_hi + tile : P.tiles + 4 * static_cast<size_t>(tile) + 3;
            atomicAdd(rows, n);
            atomicMin(plo, tlo);
            atomicMax(phi, thi);
            n = 0;
            tlo = 0xFFFFFFFFu;
            thi = 0;
        };
#pragma unroll
        for (uint32_t j = 0; j < PER; ++j) {
            if (opens >> j & 1u) {
                flush(t - 1);
                ++t;
            }
            const bool in = keys >> j & 1u;
            if (in) {
                ++n;
                tlo = tlo < lo[j] ? tlo : lo[j];
                thi = thi > hi[j] ? thi : hi[j];
            }
            own_tile = in ? t - 1 : 0xFFFFFFFFu;
            if (PER > 1 && i0 + j < P.n_tok) P.tile_of[i0 + j] = own_tile;
        }
        const uint32_t t_of_0 = __shfl_sync(0xffffffffu, t, 0);  // (every lane takes part)
        const bool one = __all_sync(0xffffffffu, n != 0 && t == t_of_0);
        if (one) {
            n = __reduce_add_sync(0xffffffffu, n);
            tlo = __reduce_min_sync(0xffffffffu, tlo);
            thi = __reduce_max_sync(0xffffffffu, thi);
            if (lane != 0) n = 0;
        }
        flush(t - 1);
        __syncthreads();  // every thread has read the carries
        if (tid == NT - 1) {
            carry_tiles += incl;
            carry_start = max_op(incl_start, before);
            last_of_slot[0] = last_slot;
            last_of_keys[0] = last_keys;
        }
        __syncthreads();
    }
    const uint32_t n_tiles = carry_tiles;
    const uint32_t kept = n_tiles < kPlanTiles ? n_tiles : kPlanTiles;
    const bool split = n_tiles <= kPlanTiles && static_cast<uint64_t>(n_tiles) * P.n_kv_head <
                                                    static_cast<uint64_t>(kSplitBelow) * P.sms;
    uint32_t ktiles = 0, rows = 0;  // of tile tid
    if (tid < kept) {
        rows = t_rows[tid];
        ktiles = (t_hi[tid] - t_lo[tid]) / BK + 1;
        if (split) t_part[tid] = ktiles;
    }
    uint32_t chunk = 0x7FFFFFFFu;
    // split s of a tile with keys lo .. hi, as list entry e
    auto put = [&](uint32_t e, uint32_t first, uint32_t n, uint32_t slot, uint32_t lo, uint32_t hi,
                   uint32_t s) {
        const uint32_t begin = lo + (s ? s * chunk * BK : 0u);
        uint32_t keys = hi - begin + 1;
        if (keys / BK >= chunk) keys = chunk * BK;
        uint4* d = reinterpret_cast<uint4*>(P.list) + 2 * static_cast<size_t>(e);
        d[0] = make_uint4(first, n, slot * P.slot_ctx + begin, begin);
        d[1] = make_uint4(keys, s, 0u, 0u);
    };
    if (split) {
        const uint32_t wmax = __reduce_max_sync(0xffffffffu, ktiles);
        if (lane == 0) atomicMax(&longest, wmax);
        __syncthreads();
        // thread s - 1 tries s splits of the longest tile; of equal costs the
        // longest chunk, so the fewest partials.  (Divisions by the chunk are
        // most of the work: a multiplication by ceil(2^32 / c) does them, exact
        // while x c < 2^32, so for tiles of fewer than 32768 key tiles.)
        if (tid < kMaxSplits) {
            const uint32_t s = tid + 1, c = (longest + s - 1) / s;
            const uint32_t magic = c > 1 && longest < 32768u ? 0xFFFFFFFFu / c + 1u : 0u;
            uint32_t items = 0;
            for (uint32_t t = 0; t < n_tiles; ++t) {
                const uint32_t x = t_part[t] + c - 1;
                items += c == 1 ? x : (magic ? __umulhi(x, magic) : x / c);
            }
            items *= P.n_kv_head;
            const uint32_t waves = (items + P.sms - 1) / P.sms;
            uint64_t cost = static_cast<uint64_t>(waves) * (c * BK + kItemCost + (s > 1 ? kItemCost / 2 : 0u));
            if (s > 1 && (c * BK < kMinChunk || items > kSplitMost * P.sms)) cost = 0x7FFFFFFFull;
            uint64_t key = (cost << 32) | (0xFFFFFFFFu - c);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const uint64_t o = __shfl_xor_sync(0xffffffffu, key, off);
                key = o < key ? o : key;
            }
            if (lane == 0) best[warp] = key;
        }
        __syncthreads();
        static_assert(kMaxSplits == 64, "two warps have a candidate a lane");
        chunk = 0xFFFFFFFFu - static_cast<uint32_t>((best[0] < best[1] ? best[0] : best[1]) & 0xFFFFFFFFu);
        const uint32_t ns = tid < n_tiles ? (ktiles + chunk - 1) / chunk : 0u;
        const uint32_t mine = ns > 1 || P.shared.lens ? ns * rows : 0u;  // partial rows
        const uint32_t base = block_inclusive(mine, scan_u, add_op, 0u) - mine;
        if (tid < n_tiles) {
            t_ns[tid] = mine ? ns : 0u;
            t_part[tid] = base;
            atomicAdd(&hist[ns], 1u);
        }
        __syncthreads();
        // split s begins in the list after the tiles with more than s' splits
        // of every s' < s; lane l has splits 2 l and 2 l + 1
        static_assert(kMaxSplits == 64, "one warp has all splits, two a lane");
        if (warp == 0) {
            auto scan = [&](uint32_t v) {
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const uint32_t o = __shfl_up_sync(0xffffffffu, v, off);
                    if (lane >= static_cast<uint32_t>(off)) v += o;
                }
                return v;
            };
            const uint32_t h0 = hist[2 * lane], h1 = hist[2 * lane + 1];
            const uint32_t upto = scan(h0 + h1);              // tiles of <= 2 l + 1 splits
            const uint32_t m1 = n_tiles - upto, m0 = m1 + h1;  // tiles that have split 2 l + 1, 2 l
            const uint32_t end = scan(m0 + m1);
            at[2 * lane] = end - m0 - m1;
            at[2 * lane + 1] = end - m1;
            if (lane == 31) at[kMaxSplits] = end;
        }
        __syncthreads();
        for (uint32_t s = 0; s < ns; ++s)
            put(atomicAdd(&at[s], 1u), t_first[tid], rows, t_slot[tid], t_lo[tid], t_hi[tid], s);
        for (uint32_t i = tid; i < P.n_tok; i += NT) {
            const uint32_t t = PER == 1 ? own_tile : P.tile_of[i];  // (one round: its own token)
            rec[2 * i] = t == 0xFFFFFFFFu || t_ns[t] == 0
                             ? make_uint4(0u, 0u, 0u, 0u)
                             : make_uint4(t_part[t] + (i - t_first[t]), t_rows[t], t_ns[t], 0u);
        }
    } else {
        for (uint32_t t = tid; t < n_tiles; t += NT) {
            const bool near = t < kPlanTiles;
            const uint4 x = near ? make_uint4(t_first[t], t_rows[t], t_slot[t], t_hi[t]) : __ldcg(tiles + t);
            put(n_tiles - 1 - t, x.x, x.y, x.z, near ? t_lo[t] : __ldcg(P.tile_lo + t), x.w, 0u);
        }
        // a shared call's unsplit rows have one partial each
        for (uint32_t i = tid; i < P.n_tok; i += NT)
            rec[2 * i] = make_uint4(
                i, 0u, P.shared.lens && (PER == 1 ? own_tile : P.tile_of[i]) != 0xFFFFFFFFu ? 1u : 0u, 0u);
    }
    if (tid == 0) {
        P.plan[0] = (split ? at[kMaxSplits] : n_tiles) * P.n_kv_head;
        P.plan[1] = P.sms;  // the CTAs' first items are theirs without asking
        P.plan[2] = split ? 1u : 0u;
    }
    // a shared call's decode plan runs before this kernel, which may have
    // started beside it: this kernel ends after it
    grid_dependency_wait();
}

template <int MT, int BK, uint32_t NT, uint32_t PER>
__global__ void __launch_bounds__(NT, 1)
    slotkv_scored_plan_kernel(const ScoredPrefillParams P) {
    // This kernel is a programmatic dependent: of the decode plan in a shared
    // call, which has waited for the work before the call, else of that work.
    if (!P.after_plan) grid_dependency_wait();
    // Prep, launched next as a programmatic dependent, may start at once: it
    // reads nothing of what this kernel writes, and its last CTA waits for
    // this kernel, so the attention kernel after it waits for both.
    grid_launch_dependents();
    scored_plan<MT, BK, NT, PER>(P);
}

// Calls of up to kFrontRows rows have the plan (CTA 0) and prep (the others) in
// one launch: such a call takes the host, at 2 to 5 us a launch, about as long
// as the GPU (six rows on a prefix 17.1 -> 16.2 us, 9 tokens on 600 keys 16.5
// -> 15.6, 51 rows on two prefixes 98.8 -> 97.9).  Larger calls keep the plan's
// 1024 threads and prep's small CTAs, which fill the SMs better.
constexpr uint32_t kFrontRows = 256, kFrontThreads = 256;
template <int HD, int MT, int BK>
__global__ void __launch_bounds__(kFrontThreads)
    slotkv_scored_front_kernel(const ScoredPrefillParams P) {
    if (!P.after_plan) grid_dependency_wait();  // (as the plan kernel)
    grid_launch_dependents();
    if (blockIdx.x == 0)
        scored_plan<MT, BK, kFrontThreads, 1>(P);
    else
        prefill_prep<HD, true>(P, (blockIdx.x - 1) * (kFrontThreads / 32) + (threadIdx.x >> 5));
}

// ------------------------------------------------------------------ attention
// Half-tile h of the CTA's stream of key tiles: h = 2g is tile g's K, h = 2g + 1
// its V; it lives in slot h % NSLOT.
template <int HD, int G, bool SC = false>
__global__ void __launch_bounds__(SC ? PCfg<HD, G, SC>::THREADS_SC : PCfg<HD, G>::THREADS, 1)
    slotkv_prefill_tc_kernel(const __grid_constant__ CUtensorMap tmK,
                             const __grid_constant__ CUtensorMap tmV,
                             const prefill_params_t<SC> P) {
    using C = PCfg<HD, G, SC>;
    constexpr int BK = C::BK, NB = C::NB, NSLOT = C::NSLOT, NBUF = C::NBUF;
    constexpr float kLog2e = 1.4426950408889634f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile uint32_t* desc = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_DESC);
    volatile uint32_t* meta = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_META);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::OFF_TSLOT);
    [[maybe_unused]] auto log_of = [&](int w) {
        return reinterpret_cast<volatile uint32_t*>(smem + C::OFF_LOG) + w * (2 * C::LOG + 2);
    };
    const uint32_t ring = smem_addr(smem);
    const uint32_t bar0 = smem_addr(smem + C::OFF_BAR);
    const uint32_t FULL = bar0, CONV = FULL + 8 * NSLOT, EMPTY = CONV + 8 * NSLOT;
    auto full_bar = [&](uint32_t h) { return FULL + 8 * (h % NSLOT); };
    auto conv_bar = [&](uint32_t h) { return CONV + 8 * (h % NSLOT); };
    auto land_phase = [](uint32_t h) { return (h / NSLOT) & 1u; };
    const uint32_t SFULL = EMPTY + 8 * NSLOT, PREADY = SFULL + 16;
    const uint32_t PVDONE = PREADY + 16, QREADY = PVDONE + 16, IFULL = QREADY + 8;
    const uint32_t IFREE = IFULL + 16, DRAIN = IFREE + 16;
    // hi and lo operand buffers of a slot
    auto slot_hi = [&](uint32_t sl) { return ring + sl * C::SLOT; };
    auto slot_lo = [&](uint32_t sl) { return ring + sl * C::SLOT + C::BUF; };

    if (tid == 0) {
        for (int i = 0; i < NSLOT; ++i) {
            mbar_init(FULL + 8 * i, 1);
            mbar_init(CONV + 8 * i, C::NCONV);
            mbar_init(EMPTY + 8 * i, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(SFULL + 8 * b, 1);
            mbar_init(PREADY + 8 * b, C::NSW);
            mbar_init(PVDONE + 8 * b, 1);
            mbar_init(IFULL + 8 * b, 1);
            mbar_init(IFREE + 8 * b, C::NSW + 1);
        }
        mbar_init(QREADY, C::NSW);
        mbar_init(DRAIN, 1);
        misc[0] = 0;
        if constexpr (SC)
            for (int w = 0; w < C::NCONV; ++w) log_of(w)[2 * C::LOG] = log_of(w)[2 * C::LOG + 1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0) {
        tc::tmem_alloc(smem_addr(tslot), C::TMEM_COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tslot;
    // (scored calls: set up beside the kernels before it)
    if constexpr (SC) grid_dependency_wait();
    auto timeout = [&]() {
        atomicOr(P.status, kDevTimeout);
        misc[0] = 1;
    };

    if (warp >= C::NSW) {
        if constexpr (SC) regs_decrease<C::REG_OTHER>();
        if (warp == C::WARP_TMA) {
            // ------------------------------------------------------------ producer
            if (lane == 0) {
                uint32_t n_items = 0;
                [[maybe_unused]] const uint4* tiles = reinterpret_cast<const uint4*>(P.tiles);
                uint32_t h = 0;  // half-tiles issued
                // wait until slot h % NSLOT is free again
                auto slot_free = [&](uint32_t hh) {
                    return hh < static_cast<uint32_t>(NSLOT) ||
                           mbar_wait(EMPTY + 8 * (hh % NSLOT), ((hh / NSLOT) - 1) & 1);
                };
                for (uint32_t k = 0;; ++k) {
                    const uint32_t is = k & 1;
                    if (k >= 2 && !mbar_wait(IFREE + 8 * is, ((k >> 1) - 1) & 1)) {
                        timeout();
                        break;
                    }
                    if (misc[0]) break;
                    volatile uint32_t* d = desc + 8 * is;
                    // scored calls: a CTA's first item is its own, and an entry
                    // has all there is to know of an item, so that the first
                    // copies start one memory latency after the plan
                    const uint32_t it = SC && k == 0 ? blockIdx.x : atomicAdd(P.plan + 1, 1u);
                    [[maybe_unused]] uint4 e0 = make_uint4(0, 0, 0, 0), e1 = e0;
                    if constexpr (SC) {
                        if (k == 0 || it < n_items) {
                            const uint4* e = reinterpret_cast<const uint4*>(P.list) +
                                             2 * static_cast<size_t>(it / P.n_kv_head);
                            e0 = __ldcg(e);
                            e1 = __ldcg(e + 1);
                        }
                    }
                    if (k == 0) n_items = __ldcg(P.plan);
                    if (it >= n_items) {
                        // nothing left for this CTA: what follows may be launched
                        if constexpr (SC) grid_launch_dependents();
                        d[6] = 1;
                        mbar_arrive(IFULL + 8 * is);
                        // tell the converters: an end marker in the next slot
                        if (!slot_free(h)) {
                            timeout();
                            break;
                        }
                        meta[4 * (h % NSLOT) + 1] = 1;
                        mbar_arrive(full_bar(h));
                        if constexpr (SC) {  // and one for the V converters
                            ++h;
                            if (!slot_free(h)) {
                                timeout();
                                break;
                            }
                            meta[4 * (h % NSLOT) + 1] = 1;
                            mbar_arrive(full_bar(h));
                        }
                        break;
                    }
                    const uint32_t kvh = it % P.n_kv_head;
                    uint32_t y_row, keys;  // first row in the [rows][kv_dim] view, keys from it
                    if constexpr (SC) {
                        y_row = e0.z;
                        keys = e1.x;
                        d[0] = e0.x;
                        d[1] = e0.y;
                        d[2] = e0.w;  // first key
                        d[3] = e1.y;  // split
                    } else {
                        // in the plan's hand-out order; keys 0 .. max_pos
                        const uint4 rec = __ldcg(tiles + __ldcg(P.tile_of + it / P.n_kv_head));
                        y_row = rec.z * P.slot_ctx;
                        keys = rec.w + 1;
                        d[0] = rec.x;
                        d[1] = rec.y;
                        d[2] = rec.z;
                        d[3] = rec.w;
                    }
                    const uint32_t ntiles = (keys + BK - 1) / BK;
                    d[4] = kvh;
                    d[5] = ntiles;
                    d[6] = 0;
                    mbar_arrive(IFULL + 8 * is);
                    const int y0 = static_cast<int>(y_row);
                    for (uint32_t t = 0; t < ntiles && !misc[0]; ++t) {
                        const uint32_t left = keys - t * BK;
                        const int y = y0 + static_cast<int>(t * BK);
                        for (int which = 0; which < 2; ++which, ++h) {  // K, then V
                            if (!slot_free(h)) {
                                timeout();
                                break;
                            }
                            const uint32_t sl = h % NSLOT;
                            meta[4 * sl + 0] = left < static_cast<uint32_t>(BK) ? left : BK;
                            meta[4 * sl + 1] = 0;
                            mbar_expect_tx(full_bar(h), C::BUF);
#pragma unroll
                            for (int c = 0; c < NB; ++c)
                                tma_load_2d(slot_hi(sl) + c * C::BLK, which ? &tmV : &tmK,
                                            static_cast<int>(kvh * HD) + 32 * c, y, full_bar(h));
                        }
                    }
                    if (misc[0]) break;
                }
                if (misc[0]) {
                    // drain this CTA's copies that may still be in flight
                    for (uint32_t u = h > static_cast<uint32_t>(NSLOT) ? h - NSLOT : 0; u < h; ++u)
                        mbar_wait(full_bar(u), land_phase(u), 1ll << 28);
                }
            }
        } else if (warp >= C::WARP_CONV + C::NCONV) {
            // ------------------------------------------------------------ K converters
            // (scored calls; the others below then only take V).  K's lo part
            // beside it, as below, with all of a thread's loads of a batch in
            // flight before its stores; no warp waits for another.
            constexpr int NT = C::NKCONV * 32, PER = C::BUF / 16 / NT, BATCH = 8;
            static_assert(PER % BATCH == 0, "whole batches");
            const int ct = tid - (C::WARP_CONV + C::NCONV) * 32;
            for (uint32_t h = 0;; h += 2) {
                const uint32_t sl = h % NSLOT;
                const bool ok = __all_sync(0xffffffffu, mbar_wait(full_bar(h), land_phase(h)));
                if (!ok) timeout();
                if (__any_sync(0xffffffffu, !ok || misc[0] || meta[4 * sl + 1])) break;
                const uint32_t rows = meta[4 * sl + 0];
                float4* hi = reinterpret_cast<float4*>(smem + sl * C::SLOT);
                float4* lo = reinterpret_cast<float4*>(smem + sl * C::SLOT + C::BUF);
#pragma unroll
                for (int b = 0; b < PER; b += BATCH) {
                    float4 x[BATCH];
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) x[j] = hi[ct + (b + j) * NT];
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) {
                        const int i = ct + (b + j) * NT;
                        const uint32_t row = static_cast<uint32_t>(i % (C::BLK / 16)) / 8;
                        if (row >= rows) {  // past the item's last key
                            x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                            hi[i] = x[j];
                        }
                        uint32_t h0, h1, h2, h3, l0, l1, l2, l3;
                        tf32_split(x[j].x, h0, l0);
                        tf32_split(x[j].y, h1, l1);
                        tf32_split(x[j].z, h2, l2);
                        tf32_split(x[j].w, h3, l3);
                        lo[i] = make_float4(__uint_as_float(l0), __uint_as_float(l1),
                                            __uint_as_float(l2), __uint_as_float(l3));
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane < C::NCONV / C::NKCONV) mbar_arrive(conv_bar(h));
            }
        } else if (warp >= C::WARP_CONV) {
            // ------------------------------------------------------------ converters
            const int ct = tid - C::WARP_CONV * 32;
            const int w = ct >> 5;
            constexpr int NT = C::NCONV * 32;
            // (scored calls: V only, the odd half-tiles)
            for (uint32_t h = SC ? 1 : 0;; h += SC ? 2 : 1) {
                const uint32_t sl = h % NSLOT;
                // The converter warps meet at named barriers below, so they must
                // all stop at the same half-tile: each publishes its own reason
                // to stop (a wait that expired, an abort, the end marker) and all
                // decide from the published flags.
                const bool ok = mbar_wait(full_bar(h), land_phase(h));
                if (!ok) timeout();
                if (lane == 0) misc[2 + w] = (!ok || misc[0] || meta[4 * sl + 1]) ? 1 : 0;
                named_sync_conv<NT>();
                int stop = 0;
#pragma unroll
                for (int w2 = 0; w2 < C::NCONV; ++w2) stop |= misc[2 + w2];
                if (stop) break;
                const uint32_t rows = meta[4 * sl + 0];
                uint8_t* hib = smem + sl * C::SLOT;
                uint8_t* lob = hib + C::BUF;
                if (!SC && (h & 1) == 0) {
                    // K: the landed f32 tile is its own hi part (the tensor core
                    // reads a TF32 operand's f32 bits with the low 13 mantissa
                    // bits ignored, i.e. as x & 0xFFFFE000), so only the lo part
                    // is written beside it (K-major, as TMA laid the tile out);
                    // rows past the item's last key are zeroed in both
                    float4* hi = reinterpret_cast<float4*>(hib);
                    float4* lo = reinterpret_cast<float4*>(lob);
#pragma unroll
                    for (int i = ct; i < C::BUF / 16; i += NT) {
                        // each 128-byte row of a column block is 8 float4s
                        const uint32_t row = static_cast<uint32_t>(i % (C::BLK / 16)) / 8;
                        if (row >= rows) {
                            hi[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                            lo[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                            continue;
                        }
                        const float4 x = hi[i];
                        uint32_t h0, h1, h2, h3, l0, l1, l2, l3;
                        tf32_split(x.x, h0, l0);
                        tf32_split(x.y, h1, l1);
                        tf32_split(x.z, h2, l2);
                        tf32_split(x.w, h3, l3);
                        lo[i] = make_float4(__uint_as_float(l0), __uint_as_float(l1),
                                            __uint_as_float(l2), __uint_as_float(l3));
                    }
                } else {
                    // V: every 32 x 32 sub-block transposed (keys along the
                    // 128-byte rows), hi in place, lo into the lo buffer.  All
                    // converter threads read their sub-blocks (lane = dim, one
                    // key per load) before any writes, so the in-place
                    // permutation is safe whatever its cycles.
                    float x[C::SB_PER_WARP][32];
#pragma unroll
                    for (int j = 0; j < C::SB_PER_WARP; ++j) {
                        const int sb = w + C::NCONV * j;
                        const int kb = sb / NB, db = sb % NB;
                        const uint8_t* src = hib + db * C::BLK + kb * 4096;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const uint32_t off = (k / 8) * 1024 + (k % 8) * 128 +
                                                 (((lane / 4) ^ (k % 8)) * 16) + (lane % 4) * 4;
                            const float v = *reinterpret_cast<const float*>(src + off);
                            x[j][k] = static_cast<uint32_t>(kb * 32 + k) < rows ? v : 0.f;
                        }
                    }
                    if constexpr (SC) {
                        // the largest magnitude's bits tell whether every value is finite
                        uint32_t top = 0;
#pragma unroll
                        for (int j = 0; j < C::SB_PER_WARP; ++j)
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const uint32_t u = __float_as_uint(x[j][k]) & 0x7FFFFFFFu;
                                top = top > u ? top : u;
                            }
                        if (__builtin_expect(__any_sync(0xffffffffu, top >= 0x7F800000u), 0)) {
                            // into the log (seen by the epilogue through this
                            // tile's barriers): the newest run goes on over a
                            // few tiles without one
                            if (lane == 0) {
                                volatile uint32_t* log = log_of(w);
                                const uint32_t g = h / 2;
                                uint32_t n = log[2 * C::LOG];
                                if (n == 0 || g > log[2 * C::LOG + 1] + C::LOG_GAP) {
                                    log[2 * (n % C::LOG)] = g;
                                    ++n;
                                }
                                log[2 * ((n - 1) % C::LOG) + 1] = g;
                                log[2 * C::LOG] = n;
                                log[2 * C::LOG + 1] = g + 1;
                            }
#pragma unroll
                            for (int j = 0; j < C::SB_PER_WARP; ++j)
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    if ((__float_as_uint(x[j][k]) & 0x7F800000u) == 0x7F800000u)
                                        x[j][k] = 0.f;
                        }
                    }
                    named_sync_conv<NT>();
#pragma unroll
                    for (int j = 0; j < C::SB_PER_WARP; ++j) {
                        const int sb = w + C::NCONV * j;
                        const int kb = sb / NB, db = sb % NB;
                        const uint32_t base = kb * C::VT_BLK + db * 4096 + (lane / 8) * 1024 +
                                              (lane % 8) * 128;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            uint32_t hh[4], ll[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) tf32_split(x[j][4 * c + e], hh[e], ll[e]);
                            const uint32_t off = base + ((c ^ (lane % 8)) * 16);
                            *reinterpret_cast<uint4*>(hib + off) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
                            *reinterpret_cast<uint4*>(lob + off) = make_uint4(ll[0], ll[1], ll[2], ll[3]);
                        }
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(conv_bar(h));
            }
        } else if (warp == C::WARP_MMA) {
            // ------------------------------------------------------------ MMA issuer
            // Plain calls: one thread runs the role.  Scored calls: the whole
            // warp does, in step, and one elected lane issues -- what an MMA
            // instruction takes (tensor memory columns, descriptors) is then
            // known to be the same in all lanes, so the compiler keeps it in
            // uniform registers instead of moving it there for each MMA
            if (SC || lane == 0) {
                const uint32_t tb = SC ? __shfl_sync(0xffffffffu, tbase, 0) : tbase;
                const bool lead = !SC || tc::elect_one();
                uint32_t g = 0;  // key tiles whose QK was issued
                bool ok = true;
                // a wait's outcome and the abort flag, the same for the whole
                // warp (the lanes meet again below, so they leave together).
                // Scored calls look at the abort flag only where a wait did
                // not find its phase complete at once: a role that has left
                // arrives no more.
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    if constexpr (SC) {
                        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
                        const bool done = mbar_wait(bar, parity) && misc[0] == 0;
                        return __all_sync(0xffffffffu, done) != 0;
                    } else {
                        return mbar_wait(bar, parity);
                    }
                };
                auto aborted = [&]() {
                    const bool a = misc[0] != 0;
                    return SC ? __any_sync(0xffffffffu, a) != 0 : a;
                };
                auto converted = [&](uint32_t hh) {
                    return wait(conv_bar(hh), land_phase(hh));
                };
                // O += P V for tile t of the item (global tile gp)
                auto issue_pv = [&](uint32_t t, uint32_t gp) {
                    const uint32_t hv = 2 * gp + 1;
                    if (!converted(hv) || !wait(PREADY + 8 * (gp & 1), (gp >> 1) & 1)) {
                        timeout();
                        return false;
                    }
                    tc::fence_after_sync();
                    const uint32_t sl = hv % NSLOT;
                    const uint32_t pcol0 = C::C_S + (gp % NBUF) * C::C_BUF;
                    if constexpr (SC) {
                        // the tile's own O: products with a low part first
                        const uint32_t ocol = tb + (C::TWO_O && (gp & 1) ? C::C_O2 : C::C_O);
                        const uint32_t phi = tb + pcol0, plo = phi + BK;
                        const uint64_t bh = tc::smem_desc(slot_hi(sl), 16, 1024, tc::kSwizzle128B);
                        const uint64_t bl = tc::smem_desc(slot_lo(sl), 16, 1024, tc::kSwizzle128B);
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < BK / 8; ++kk) {
                                const uint32_t off = ((kk / 4) * C::VT_BLK + (kk % 4) * 32) >> 4;
                                tc::mma_tf32_ts(ocol, plo + kk * 8, bh + off, C::IDESC_PV, kk != 0 ? 1u : 0u);
                                tc::mma_tf32_ts(ocol, phi + kk * 8, bl + off, C::IDESC_PV, 1u);
                            }
#pragma unroll
                            for (int kk = 0; kk < BK / 8; ++kk) {
                                const uint32_t off = ((kk / 4) * C::VT_BLK + (kk % 4) * 32) >> 4;
                                tc::mma_tf32_ts(ocol, phi + kk * 8, bh + off, C::IDESC_PV, 1u);
                            }
                        }
                    } else {
                        // O += P_lo V_hi + P_hi V_hi + P_hi V_lo, K-step by K-step
                        // (consecutive products share their B, then their A, slice)
#pragma unroll
                        for (int kk = 0; kk < BK / 8; ++kk) {
                            const uint32_t off = (kk / 4) * C::VT_BLK + (kk % 4) * 32;
                            const uint64_t bh = tc::smem_desc(slot_hi(sl) + off, 16, 1024, tc::kSwizzle128B);
                            const uint64_t bl = tc::smem_desc(slot_lo(sl) + off, 16, 1024, tc::kSwizzle128B);
                            tc::mma_tf32_ts(tbase + C::C_O, tbase + pcol0 + BK + kk * 8, bh, C::IDESC_PV,
                                            (t | kk) != 0 ? 1u : 0u);
                            tc::mma_tf32_ts(tbase + C::C_O, tbase + pcol0 + kk * 8, bh, C::IDESC_PV, 1u);
                            tc::mma_tf32_ts(tbase + C::C_O, tbase + pcol0 + kk * 8, bl, C::IDESC_PV, 1u);
                        }
                    }
                    if (lead) {
                        tc::mma_commit(PVDONE + 8 * (gp & 1));
                        tc::mma_commit(EMPTY + 8 * sl);
                    }
                    __syncwarp(SC ? 0xffffffffu : 1u);
                    return true;
                };
                for (uint32_t k = 0; ok; ++k) {
                    const uint32_t is = k & 1;
                    if (!wait(IFULL + 8 * is, (k >> 1) & 1)) {
                        timeout();
                        break;
                    }
                    uint32_t ntiles = desc[8 * is + 5], end = desc[8 * is + 6];
                    if constexpr (SC) {
                        ntiles = __shfl_sync(0xffffffffu, ntiles, 0);
                        end = __shfl_sync(0xffffffffu, end, 0);
                    }
                    if (lead) mbar_arrive(IFREE + 8 * is);
                    if (end || aborted()) break;
                    if (!wait(QREADY, k & 1)) {
                        timeout();
                        break;
                    }
                    tc::fence_after_sync();
                    for (uint32_t t = 0; t < ntiles; ++t, ++g) {
                        const uint32_t hk = 2 * g;
                        if (!converted(hk)) {
                            timeout();
                            ok = false;
                            break;
                        }
                        if (!SC && aborted()) {
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t sl = hk % NSLOT;
                        const uint32_t scol = C::C_S + (g % NBUF) * C::C_BUF;
                        if constexpr (SC) {
                            // S: products with a low part first, the high ones last
                            const uint64_t bh = tc::smem_desc(slot_hi(sl), 16, 1024, tc::kSwizzle128B);
                            const uint64_t bl = tc::smem_desc(slot_lo(sl), 16, 1024, tc::kSwizzle128B);
                            if (lead) {
#pragma unroll
                                for (int kk = 0; kk < HD / 8; ++kk) {
                                    const uint32_t off = ((kk / 4) * C::BLK + (kk % 4) * 32) >> 4;
                                    tc::mma_tf32_ts(tb + scol, tb + C::C_QLO + kk * 8, bh + off, C::IDESC_QK,
                                                    kk != 0 ? 1u : 0u);
                                    tc::mma_tf32_ts(tb + scol, tb + C::C_QHI + kk * 8, bl + off, C::IDESC_QK, 1u);
                                }
#pragma unroll
                                for (int kk = 0; kk < HD / 8; ++kk) {
                                    const uint32_t off = ((kk / 4) * C::BLK + (kk % 4) * 32) >> 4;
                                    tc::mma_tf32_ts(tb + scol, tb + C::C_QHI + kk * 8, bh + off, C::IDESC_QK, 1u);
                                }
                            }
                        } else {
                            // S = Q_lo K_hi + Q_hi K_hi + Q_hi K_lo, K-step by K-step
                            // (consecutive products share their B, then their A, slice)
#pragma unroll
                            for (int kk = 0; kk < HD / 8; ++kk) {
                                const uint32_t off = (kk / 4) * C::BLK + (kk % 4) * 32;
                                const uint64_t bh = tc::smem_desc(slot_hi(sl) + off, 16, 1024, tc::kSwizzle128B);
                                const uint64_t bl = tc::smem_desc(slot_lo(sl) + off, 16, 1024, tc::kSwizzle128B);
                                tc::mma_tf32_ts(tbase + scol, tbase + C::C_QLO + kk * 8, bh, C::IDESC_QK,
                                                kk != 0 ? 1u : 0u);
                                tc::mma_tf32_ts(tbase + scol, tbase + C::C_QHI + kk * 8, bh, C::IDESC_QK, 1u);
                                tc::mma_tf32_ts(tbase + scol, tbase + C::C_QHI + kk * 8, bl, C::IDESC_QK, 1u);
                            }
                        }
                        // (the failure-path test option withholds the CTA's first
                        // score-ready signal, so the softmax's bounded wait runs out)
                        if (lead) {
                            if (!(g == 0 && (P.flags & kOptTestStall))) tc::mma_commit(SFULL + 8 * (g & 1));
                            tc::mma_commit(EMPTY + 8 * sl);  // K slot free once QK has read it
                        }
                        __syncwarp(SC ? 0xffffffffu : 1u);
                        // one buffer: this tile's PV next; two: the previous tile's
                        if (NBUF == 1) {
                            if (!issue_pv(t, g)) {
                                ok = false;
                                break;
                            }
                        } else if (t >= 1 && !issue_pv(t - 1, g - 1)) {
                            ok = false;
                            break;
                        }
                    }
                    if (NBUF == 2 && ok && ntiles && !aborted() && !issue_pv(ntiles - 1, g - 1)) ok = false;
                }
                // every MMA issued above has completed before tensor memory is freed
                if (lead) tc::mma_commit(DRAIN);
                mbar_wait(DRAIN, 0, 1ll << 28);
            }
        }
    } else {
        if constexpr (SC) regs_increase<C::REG_SOFTMAX>();
        // ------------------------------------------------------------ softmax
        // Warps q and q + 4 share tensor-memory lane quarter q (rows 32 q ..
        // 32 q + 31); half hf = warp / 4 takes columns [hf BK/2, (hf+1) BK/2)
        // of each score tile and columns [hf HD/2, (hf+1) HD/2) of Q and O.
        // The two halves of a row meet at a pairwise named barrier to combine
        // their maxima (every tile) and their sums (at an item's end); both
        // keep the same running max.  Every exit from the loops is decided
        // at one of these meetings from both halves' published state (a
        // failed bounded wait or the CTA's abort flag is published, never
        // acted on alone), so neither half can leave its partner waiting at
        // the barrier.
        constexpr int HB = BK / 2, HH = HD / 2;
        static_assert((HB == 32 || HB == 16) && HH % 32 == 0, "one access per half of a score tile");
        const int quarter = warp & 3, hf = warp >> 2;
        const uint32_t r = static_cast<uint32_t>(quarter * 32 + lane);  // query row = TMEM lane
        const uint32_t lrow = tbase + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_local = r / G, h_local = r % G;
        float* xmax = reinterpret_cast<float*>(smem + C::OFF_XCH);   // [2 parities][2][M]
        float* xsum = xmax + 4 * C::M;                               // [2][M]
        int* xflag = reinterpret_cast<int*>(xmax + 6 * C::M);       // beside each value
        auto pair_sync = [&]() {
            asm volatile("bar.sync %0, 64;" ::"r"(3 + quarter) : "memory");
        };
        // Meet, and return whether any of the pair's 64 threads says so.
        [[maybe_unused]] auto pair_any = [&](bool x) {
            uint32_t any;
            asm volatile(
                "{\n\t.reg .pred P, Q;\n\tsetp.ne.u32 P, %1, 0;\n\t"
                "bar.red.or.pred Q, %2, 64, P;\n\tselp.u32 %0, 1, 0, Q;\n\t}"
                : "=r"(any)
                : "r"(x ? 1u : 0u), "r"(3 + quarter)
                : "memory");
            return any != 0;
        };
        // Publish v and this warp's stop flag (any lane's) in slot [hf][r] of
        // buf, meet, and return the partner's value; stop becomes the pair's
        // decision (either warp's flag), the same in all 64 threads.
        auto exchange = [&](float* buf, float v, bool& stop) {
            const int at = static_cast<int>(buf - xmax);
            stop = __any_sync(0xffffffffu, stop);
            buf[hf * C::M + r] = v;
            xflag[at + hf * C::M + r] = stop ? 1 : 0;
            pair_sync();
            stop = stop || xflag[at + (1 - hf) * C::M + r] != 0;
            return buf[(1 - hf) * C::M + r];
        };
        uint32_t g = 0;  // key tiles processed
        constexpr int ND = SC ? 7 : 5;
        // Meeting 1 opens item k: both halves hold its descriptor (xsum is
        // free: every meeting on it is followed by a pair barrier).  stop
        // carries a failure not yet published and becomes the pair's
        // decision; on success the descriptor's slot is released.
        auto open_item = [&](uint32_t k, bool stop, uint32_t (&d)[ND]) {
            const uint32_t is = k & 1;
            stop = stop || misc[0];
            if (!stop && !mbar_wait(IFULL + 8 * is, (k >> 1) & 1)) {
                timeout();
                stop = true;
            }
            exchange(xsum, 0.f, stop);
            if (stop) return false;
            d[0] = desc[8 * is + 0];  // first token
            d[1] = desc[8 * is + 1];  // tokens
            d[2] = desc[8 * is + 4];  // kv head
            d[3] = desc[8 * is + 5];  // key tiles
            d[4] = desc[8 * is + 6];  // end marker
            if constexpr (SC) {
                d[5] = desc[8 * is + 2];  // first key
                d[6] = desc[8 * is + 3];  // split
            }
            pair_sync();  // both have read meeting 1 before xsum is written again
            __syncwarp();
            if (lane == 0) mbar_arrive(IFREE + 8 * is);
            return true;
        };
        struct ItemRow {
            bool valid;
            uint32_t tok, pos, head;
            uint32_t lo, hi;  // scored calls: the row's keys (none: lo > hi)
            uint4 part;       // and its partials' record
        };
        auto row_of = [&](const uint32_t (&d)[ND]) {
            ItemRow w;
            w.valid = r < static_cast<uint32_t>(C::ROWS) && t_local < d[1];
            w.tok = d[0] + t_local;
            w.head = d[2] * G + h_local;
            if constexpr (SC) {
                const uint4* r8 = reinterpret_cast<const uint4*>(P.part.rec) + 2 * w.tok;
                const uint4 x = w.valid ? __ldcg(r8 + 1) : make_uint4(0u, 1u, 0u, 0u);
                w.part = w.valid ? __ldcg(r8) : make_uint4(0u, 0u, 0u, 0u);
                w.pos = x.x;
                w.lo = x.y;
                w.hi = x.z;
            } else {
                w.pos = w.valid ? __ldg(P.positions + w.tok) : 0u;
            }
            return w;
        };
        // this half of the item's q rows into tensor memory, split hi / lo
        // Scored calls stage q and out rows through 2 KB of shared memory per
        // warp, 32 rows x 16 columns at a time, rows of 64 bytes with their
        // four chunks rotated: lanes then move whole 64-byte pieces of rows
        // to and from memory, four lanes a row.  (A thread reading or writing
        // its own row touches 32 lines per instruction, which cost 7 us of q
        // and 3 of out per item.)
        [[maybe_unused]] float4* stage = reinterpret_cast<float4*>(smem + C::OFF_STAGE) + warp * 128;
        [[maybe_unused]] auto stage_at = [&](int row, int chunk) { return row * 4 + ((chunk + (row >> 1)) & 3); };
        [[maybe_unused]] auto load_q_staged = [&](const uint32_t (&d)[ND]) {
            const int sub = lane >> 2, ch = lane & 3;  // row of eight, chunk
            const float* src[4];                       // rows sub, sub + 8, ..
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t rr = static_cast<uint32_t>(quarter * 32 + i * 8 + sub);
                const bool in = rr < static_cast<uint32_t>(C::ROWS) && rr / G < d[1];
                src[i] = in ? P.q_rot + (static_cast<size_t>(d[0] + rr / G) * P.n_head + d[2] * G + rr % G) * HD +
                                  hf * HH + ch * 4
                            : nullptr;
            }
#pragma unroll
            for (int c0 = 0; c0 < HH; c0 += 32) {
                float4 x[8];  // 32 columns in flight
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = src[j & 3] ? __ldcg(reinterpret_cast<const float4*>(src[j & 3] + c0 + (j >> 2) * 16))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) stage[stage_at(i * 8 + sub, ch)] = x[p * 4 + i];
                    __syncwarp();
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float4 y = stage[stage_at(lane, c)];
                        tf32_split_rn2(y.x, y.y, hi[4 * c], hi[4 * c + 1], lo[4 * c], lo[4 * c + 1]);
                        tf32_split_rn2(y.z, y.w, hi[4 * c + 2], hi[4 * c + 3], lo[4 * c + 2], lo[4 * c + 3]);
                    }
                    tc::tmem_st16(lrow + C::C_QHI + hf * HH + c0 + p * 16, hi);
                    tc::tmem_st16(lrow + C::C_QLO + hf * HH + c0 + p * 16, lo);
                }
            }
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(QREADY);
        };
        auto load_q = [&](const ItemRow& w) {
            const float* qrow = P.q_rot + (static_cast<size_t>(w.valid ? w.tok : 0) * P.n_head + w.head) * HD;
#pragma unroll
            for (int c0 = hf * HH; c0 < (hf + 1) * HH; c0 += 32) {
                uint32_t hi[32], lo[32];
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float4 x = w.valid ? __ldcg(reinterpret_cast<const float4*>(qrow + c0 + c))
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
                    tf32_split(x.x, hi[c + 0], lo[c + 0]);
                    tf32_split(x.y, hi[c + 1], lo[c + 1]);
                    tf32_split(x.z, hi[c + 2], lo[c + 2]);
                    tf32_split(x.w, hi[c + 3], lo[c + 3]);
                }
                tc::tmem_st32(lrow + C::C_QHI + c0, hi);
                tc::tmem_st32(lrow + C::C_QLO + c0, lo);
            }
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(QREADY);
        };
        // Scored calls: this half's columns of O for its row, in registers.
        // Key tile j's own O (from global tile j's PV) is added once PV(j) has
        // completed; c is the correction of the running max since P(j).
        [[maybe_unused]] float acc[SC ? HH : 1];
        [[maybe_unused]] auto add_o = [&](int c0, const uint32_t (&v)[32], float c) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const int at = SC ? c0 + i : 0, at1 = SC ? c0 + i + 1 : 0;
                const float2 a = __ffma2_rn(
                    make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])),
                    make_float2(c, c), make_float2(acc[at], acc[at1]));
                acc[at] = a.x;
                acc[at1] = a.y;
            }
        };
        [[maybe_unused]] auto add_tile = [&](uint32_t j, float c) {
            if (!mbar_wait(PVDONE + 8 * (j & 1), (j >> 1) & 1)) {
                timeout();
                return false;
            }
            tc::fence_after_sync();
            const uint32_t ocol = C::TWO_O && (j & 1) ? C::C_O2 : C::C_O;
#pragma unroll
            for (int c0 = 0; c0 < HH; c0 += 32) {
                uint32_t v[32];
                tc::tmem_ld32(lrow + ocol + hf * HH + c0, v);
                tc::tmem_ld_wait();
                add_o(c0, v, c);
            }
            return true;
        };
        // Scored calls: 32 columns (from c0 on) of the V values that are not
        // finite, in the tiles of a converter's log that are the item's, added
        // to acc where the row attends them.  Adding one twice, or looking at a
        // tile that has none, changes nothing, so a run may hold more than its
        // tiles: those of other items, or once runs of this item may have left
        // the log (the converters are three tiles ahead at most) all before.
        [[maybe_unused]] auto add_logged = [&](volatile const uint32_t* log, const ItemRow& w, uint32_t g0,
                                               uint32_t ntiles, uint32_t k_begin, int c0) {
            const uint32_t slot = __ldg(P.slots + w.tok);
            const float* v0 = P.V + (static_cast<size_t>(slot) * P.slot_ctx * P.n_kv_head + w.head / G) * HD +
                              hf * HH + c0;
            const uint32_t n = log[2 * C::LOG];
#pragma unroll 1
            for (uint32_t i = 1; i <= n && i <= C::LOG - 4; ++i) {  // newest first
                const uint32_t last = log[2 * ((n - i) % C::LOG) + 1];
                uint32_t first = log[2 * ((n - i) % C::LOG)];
                if (last < g0) break;
                if (first < g0 || i == C::LOG - 4) first = g0;
                uint32_t key = k_begin + (first - g0) * BK;
                uint32_t end = k_begin + (last - g0 < ntiles ? last - g0 + 1 : ntiles) * BK;  // past its keys
                key = key > w.lo ? key : w.lo;
                end = end <= w.hi ? end : w.hi + 1;
#pragma unroll 1
                for (; key < end; ++key) {
                    const float4* vr = reinterpret_cast<const float4*>(
                        v0 + static_cast<size_t>(key) * P.n_kv_head * HD);
                    auto add = [&](int at, float x) {
                        if ((__float_as_uint(x) & 0x7F800000u) == 0x7F800000u) acc[at] += x;
                    };
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float4 x = vr[c];
                        const int at = SC ? c0 + 4 * c : 0;
                        add(at, x.x);
                        add(at + 1, x.y);
                        add(at + 2, x.z);
                        add(at + 3, x.w);
                    }
                }
            }
        };
        [[maybe_unused]] CapSeries cap_k{};
        if constexpr (SC) cap_k = cap_series(P.rule.cap_in);
        uint32_t d[ND];
        if (open_item(0, false, d) && !d[4]) {
            ItemRow cur = row_of(d);
            if constexpr (SC) load_q_staged(d);
            else load_q(cur);
            for (uint32_t k = 0;; ++k) {
                const uint32_t ntiles = d[3];
                [[maybe_unused]] uint32_t k_begin = 0, split = 0;
                [[maybe_unused]] float slope2 = 0.f;
                if constexpr (SC) {
                    k_begin = d[5];
                    split = d[6];
                    if (P.rule.slopes) slope2 = __ldg(P.rule.slopes + cur.head) * kRuleLog2e;
                }
                float m = -CUDART_INF_F, l = 0.f;  // l: this half's share of the row sum
                bool failed = false;
                [[maybe_unused]] float corr_prev = 1.f;  // the last tile's correction of the max
                if constexpr (SC) {
#pragma unroll
                    for (int i = 0; i < HH; ++i) acc[i] = 0.f;
                }
                for (uint32_t t = 0; t < ntiles; ++t, ++g) {
                    if (!mbar_wait(SFULL + 8 * (g & 1), (g >> 1) & 1)) {
                        timeout();
                        failed = true;
                    }
                    tc::fence_after_sync();
                    const uint32_t scol = C::C_S + (g % NBUF) * C::C_BUF + hf * HB;
                    float s[HB];
                    {
                        uint32_t v[HB];
                        tc::tmem_ld(lrow + scol, v);
                        if constexpr (SC && C::TWO_O) {
                            // two: the O of tile t - 2 with S(t), whose commit
                            // covers its PV
                            static_assert(!C::TWO_O || HH == 32, "one access per half of O");
                            if (t >= 2) {
                                uint32_t o[32];
                                tc::tmem_ld32(lrow + (g & 1 ? C::C_O2 : C::C_O) + hf * HH, o);
                                tc::tmem_ld_wait();
                                add_o(0, o, corr_prev);
                            }
                        }
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < HB; ++c) s[c] = __uint_as_float(v[c]);
                    }
                    // causal mask: key kbase + c is attended iff it is <= cur.pos
                    uint32_t kbase = t * BK + hf * HB;
                    float mx = -CUDART_INF_F;
                    if constexpr (SC) {
                        kbase += k_begin;
                        if (P.rule.cap_out != 0.f) cap_scores(s, P.rule, cap_k);
                        if (P.rule.slopes) {
                            const float d0 = static_cast<float>(static_cast<int>(cur.pos - kbase));
#pragma unroll
                            for (int c = 0; c < HB; ++c)
                                s[c] = fmaf(-slope2, fabsf(d0 - static_cast<float>(c)), s[c]);
                        }
                        if (kbase < cur.lo || kbase + HB - 1 > cur.hi) {
#pragma unroll
                            for (int c = 0; c < HB; ++c) {
                                const uint32_t key = kbase + static_cast<uint32_t>(c);
                                s[c] = key >= cur.lo && key <= cur.hi ? s[c] : -CUDART_INF_F;
                            }
                        }
                        float m4[4] = {s[0], s[1], s[2], s[3]};  // four short chains
#pragma unroll
                        for (int c = 4; c < HB; ++c) m4[c & 3] = fmaxf(m4[c & 3], s[c]);
                        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    } else if (kbase + HB - 1 <= cur.pos) {
#pragma unroll
                        for (int c = 0; c < HB; ++c) mx = fmaxf(mx, s[c]);
                    } else {
#pragma unroll
                        for (int c = 0; c < HB; ++c) {
                            s[c] = kbase + static_cast<uint32_t>(c) <= cur.pos ? s[c] : -CUDART_INF_F;
                            mx = fmaxf(mx, s[c]);
                        }
                    }
                    // meeting 2 (every tile): the row's max over both halves
                    // (double-buffered by tile parity: a half writes parity p
                    // again only after the next meeting, which its partner
                    // reaches after reading p)
                    bool stop2 = failed || misc[0];
                    // (scored calls: the values are exchanged only when some
                    // row of the pair would raise its max, or to stop)
                    if (!SC || pair_any(stop2 || mx > m + 8.f)) {
                        const float other = exchange(xmax + (g & 1) * 2 * C::M, mx, stop2);
                        if (stop2) {
                            failed = true;
                            break;
                        }
                        mx = fmaxf(mx, other);
                    }
                    // lazy running max: raised only when a score passes it by 2^8
                    float corr = 1.f;
                    bool rescale = false;
                    if (mx > m + 8.f) {
                        corr = m == -CUDART_INF_F ? 0.f : fast_exp2(m - mx);
                        rescale = t > 0;
                        l *= corr;
                        m = mx;
                    }
                    if constexpr (SC) {
                        // (a row without a key so far: every score is -inf, every weight 0)
                        const float m0 = m == -CUDART_INF_F ? 0.f : m;
                        const float2 mm = make_float2(-m0, -m0);
                        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < HB; c += 2) {
                            const float2 x = __fadd2_rn(make_float2(s[c], s[c + 1]), mm);
                            s[c] = fast_exp2(x.x);
                            s[c + 1] = fast_exp2(x.y);
                            l2[(c >> 1) & 1] = __fadd2_rn(l2[(c >> 1) & 1], make_float2(s[c], s[c + 1]));
                        }
                        l += (l2[0].x + l2[1].x) + (l2[0].y + l2[1].y);
                    } else {
#pragma unroll
                        for (int c = 0; c < HB; ++c) {
                            s[c] = s[c] == -CUDART_INF_F ? 0.f : fast_exp2(s[c] - m);
                            l += s[c];
                        }
                    }
                    if constexpr (SC) {
                        // O is in registers; the tile whose O is still to be
                        // read takes the correction then
                        if (rescale) {
#pragma unroll
                            for (int i = 0; i < HH; ++i) acc[i] *= corr;
                        }
                        corr_prev = rescale ? corr : 1.f;
                        // two score buffers but one O: that of tile t - 1 is read
                        // before P(t) lets the tensor core write it again
                        if constexpr (!C::TWO_O) {
                            if (t >= 1 && !add_tile(g - 1, corr_prev)) failed = true;
                        }
                    }
                    // O may be rescaled only once the previous tile's O += P V
                    // (global tile g - 1) has completed.  PV(j) completes a phase
                    // of pv_done[j % 2]; at any wait for PV(j), PV(j - 2) has
                    // completed (the S this softmax already read was committed
                    // after it) and PV(j + 2) cannot start (it needs P from this
                    // softmax), so the parity of phase j / 2 is unambiguous.
                    // (One barrier for all PVs would not do: with two score
                    // buffers PV(j - 1) may still be running at the wait for
                    // PV(j), and its parity would read as already complete.)
                    // Both halves of a row take the same decision; a wait that
                    // runs out is published at the next meeting.
                    if (!SC && __any_sync(0xffffffffu, rescale)) {
                        if (!mbar_wait(PVDONE + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1)) {
                            timeout();
                            failed = true;
                        } else {
                            tc::fence_after_sync();
#pragma unroll
                            for (int c0 = hf * HH; c0 < (hf + 1) * HH; c0 += 32) {
                                uint32_t v[32];
                                tc::tmem_ld32(lrow + C::C_O + c0, v);
                                tc::tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < 32; ++c)
                                    v[c] = __float_as_uint(__uint_as_float(v[c]) * corr);
                                tc::tmem_st32(lrow + C::C_O + c0, v);
                            }
                        }
                    }
                    {
                        uint32_t hi[HB], lo[HB];
#pragma unroll
                        for (int c = 0; c < HB; c += 2) {
                            if constexpr (SC) {
                                tf32_split_rn2(s[c], s[c + 1], hi[c], hi[c + 1], lo[c], lo[c + 1]);
                            } else {
                                tf32_split(s[c], hi[c], lo[c]);
                                tf32_split(s[c + 1], hi[c + 1], lo[c + 1]);
                            }
                        }
                        tc::tmem_st(lrow + scol, hi);
                        tc::tmem_st(lrow + scol + BK, lo);
                    }
                    tc::tmem_st_wait();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(PREADY + 8 * (g & 1));
                }
                // The next item opens before this one ends: every QK of this
                // item has completed (its last S was read above), so the next
                // item's Q may replace this one's in tensor memory while the
                // last O += P V runs, and the next item's first QK overlaps
                // this item's epilogue.  Its first O += P V overwrites O only
                // after its P is published, which this softmax does after
                // reading O below.  A failure so far is published at this
                // meeting, and both halves leave together.
                if (!open_item(k + 1, failed, d)) break;
                const bool last = d[4] != 0;
                ItemRow nxt{};
                if (!last) {
                    nxt = row_of(d);
                    if constexpr (SC) load_q_staged(d);
                    else load_q(nxt);
                }
                // This item's last O += P V (global tile g - 1; its commit
                // covers every earlier MMA), then out = O / l (both halves'
                // sums, sink included).  Meeting 3, the sums, publishes a
                // wait that ran out.
                bool stop3;
                if constexpr (SC) {
                    stop3 = C::TWO_O && ntiles >= 2 && !add_tile(g - 2, corr_prev);
                    stop3 = !add_tile(g - 1, 1.f) || stop3;
                } else {
                    stop3 = !mbar_wait(PVDONE + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1);
                    if (stop3) timeout();
                }
                const float l_other = exchange(xsum, l, stop3);
                pair_sync();  // both have read the sums before xsum is written again
                if (stop3) break;
                tc::fence_after_sync();
                const float lt = l + l_other;
                float f = 1.f / lt;
                float* orow = P.out + (static_cast<size_t>(cur.tok) * P.n_head + cur.head) * HD;
                bool direct = true;  // the row's output, not a split's partial
                if constexpr (SC) {
                    if (cur.valid) {
                        const uint4 rec = cur.part;
                        if (rec.z != 0u) {
                            direct = false;
                            f = 1.f;
                            const size_t prow = (static_cast<size_t>(rec.x) +
                                                 static_cast<size_t>(split) * rec.y) *
                                                    P.n_head + cur.head;
                            orow = P.part.acc + prow * HD;
                            if (hf == 0)
                                reinterpret_cast<float2*>(P.part.ml)[prow] = make_float2(m, lt);
                        } else if (m == -CUDART_INF_F) {
                            direct = false;
                            f = 0.f;  // no key: zeros
                        }
                    }
                }
                if (direct && P.sinks) {
                    const float sk = __ldg(P.sinks + cur.head) * kLog2e;
                    const float M2 = fmaxf(m, sk);
                    const float c = exp2f(m - M2);
                    f = c / (lt * c + exp2f(sk - M2));
                }
                if constexpr (SC) {
                    // the values the tensor core took as 0, for the keys of
                    // this item that the row attends
                    const uint32_t g0 = g - ntiles;  // the item's first tile
                    // the two converter warps whose dims are in this half
                    volatile uint32_t* log0 = log_of(NB == 4 ? 2 * hf : hf);
                    volatile uint32_t* log1 = log_of(NB == 4 ? 2 * hf + 1 : hf + 2);
                    const bool met = log0[2 * C::LOG + 1] > g0 || log1[2 * C::LOG + 1] > g0;
                    if (__builtin_expect(met && cur.valid, 0)) {
                        add_logged(log0, cur, g0, ntiles, k_begin, 0);
                        add_logged(log1, cur, g0, ntiles, k_begin, NB == 4 ? 32 : 0);
                    }
                    // rows to memory by way of the stage; each lane has the
                    // destinations of the four rows it writes pieces of
                    const int sub = lane >> 2, ch = lane & 3;
                    const uint64_t mine = cur.valid ? reinterpret_cast<uint64_t>(orow) : 0ull;
                    float* dst[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        dst[i] = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, mine, i * 8 + sub));
                        if (dst[i]) dst[i] += hf * HH + ch * 4;
                    }
#pragma unroll
                    for (int c0 = 0; c0 < HH; c0 += 16) {
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            stage[stage_at(lane, c)] =
                                make_float4(acc[c0 + 4 * c] * f, acc[c0 + 4 * c + 1] * f,
                                            acc[c0 + 4 * c + 2] * f, acc[c0 + 4 * c + 3] * f);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 y = stage[stage_at(i * 8 + sub, ch)];
                            // (streaming: q's rows stay in L2 for the items to come)
                            if (dst[i]) __stcs(reinterpret_cast<float4*>(dst[i] + c0), y);
                        }
                    }
                } else {
#pragma unroll
                    for (int c0 = hf * HH; c0 < (hf + 1) * HH; c0 += 32) {
                        uint32_t v[32];
                        tc::tmem_ld32(lrow + C::C_O + c0, v);
                        tc::tmem_ld_wait();
                        if (cur.valid) {
#pragma unroll
                            for (int c = 0; c < 32; c += 4)
                                *reinterpret_cast<float4*>(orow + c0 + c) =
                                    make_float4(__uint_as_float(v[c]) * f, __uint_as_float(v[c + 1]) * f,
                                                __uint_as_float(v[c + 2]) * f, __uint_as_float(v[c + 3]) * f);
                        }
                    }
                }
                tc::fence_before_sync();
                if (last) break;
                cur = nxt;
            }
        }
    }
    // ---------------------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tbase, C::TMEM_COLS);
}

// Join the splits of one (token, head) of a scored prefill, by one warp,
// splits in order.
template <int HD>
__device__ __forceinline__ void combine_row(const ScoredPrefillParams& P, uint4 rec, uint32_t tok,
                                            uint32_t head, uint32_t lane) {
    const size_t at0 = static_cast<size_t>(rec.x) * P.n_head + head;
    const size_t step = static_cast<size_t>(rec.y) * P.n_head;
    constexpr int EL = HD / 32;  // elements per lane
    float v[4][EL];
    auto load4 = [&](uint32_t s0) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2* src = reinterpret_cast<const float2*>(P.part.acc + (at0 + (s0 + u) * step) * HD);
#pragma unroll
            for (int e = 0; e < EL / 2; ++e) {
                const float2 x = s0 + u < rec.z ? __ldcg(src + lane + 32 * e) : make_float2(0.f, 0.f);
                v[u][2 * e] = x.x;
                v[u][2 * e + 1] = x.y;
            }
        }
    };
    load4(0);  // (in flight with the maxima and sums)
    // lanes take splits lane and lane + 32 (kMaxSplits is 64)
    float2 c[2];
    float M = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t s = lane + 32 * j;
        c[j] = s < rec.z ? __ldcg(reinterpret_cast<const float2*>(P.part.ml) + at0 + s * step)
                         : make_float2(-CUDART_INF_F, 0.f);
        M = fmaxf(M, c[j].x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float w[2], L = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        w[j] = partial_weight(c[j].x, M);
        L = __fmaf_rn(c[j].y, w[j], L);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    float f = 1.f / L;
    if (M == -CUDART_INF_F) {
        f = 0.f;  // no key: zeros
    } else if (P.sinks) {
        const float sk = __ldg(P.sinks + head) * kRuleLog2e;
        const float M2 = fmaxf(M, sk);
        const float cm = exp2f(M - M2);
        f = cm / (L * cm + exp2f(sk - M2));
    }
    float a[EL] = {};
    for (uint32_t s0 = 0; s0 < rec.z; s0 += 4) {
        if (s0) load4(s0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t s = s0 + u;
            const float wu = __shfl_sync(0xffffffffu, s < 32 ? w[0] : w[1], s & 31);
#pragma unroll
            for (int e = 0; e < EL; ++e) a[e] = __fmaf_rn(wu, v[u][e], a[e]);
        }
    }
    float2* o = reinterpret_cast<float2*>(P.out + (static_cast<size_t>(tok) * P.n_head + head) * HD);
#pragma unroll
    for (int e = 0; e < EL / 2; ++e) o[lane + 32 * e] = make_float2(a[2 * e] * f, a[2 * e + 1] * f);
}

// Every prefill launches it: whether the plan split the tiles is known on the
// device alone, since rows out of range belong to no tile (a padded call may
// have few).  With nothing to join its CTAs end at once, ~1.5 us of a call's
// end.  517 tokens of 64 heads of 64 in four splits: 13 us after the attention
// kernel's end (34 MB read, 8 MB written: 3.3 TB/s), one round trip per row
// for its partials; 24 us at four CTAs per SM.
constexpr uint32_t kCombineCtas = 16;
template <int HD>
__global__ void __launch_bounds__(128) slotkv_combine_kernel(const ScoredPrefillParams P) {
    grid_dependency_wait();
    grid_launch_dependents();
    if (__ldcg(P.plan + 2) == 0u) return;
    // a warp's rows are one grid apart; its lanes look up which of the next 32
    // have splits (rows that the attention kernel has finished itself have none)
    const uint32_t n = P.n_tok * P.n_head, warps = gridDim.x * 4, lane = threadIdx.x & 31;
    for (uint64_t w0 = blockIdx.x * 4 + (threadIdx.x >> 5); w0 < n; w0 += 32ull * warps) {
        const uint64_t mine = w0 + static_cast<uint64_t>(lane) * warps;
        uint4 rec = make_uint4(0, 0, 0, 0);
        if (mine < n)
            rec = __ldcg(reinterpret_cast<const uint4*>(P.part.rec) +
                         2 * static_cast<size_t>(static_cast<uint32_t>(mine) / P.n_head));
        for (uint32_t left = __ballot_sync(0xffffffffu, rec.z != 0u); left; left &= left - 1) {
            const int from = __ffs(left) - 1;
            const uint32_t w = static_cast<uint32_t>(w0) + from * warps;
            const uint4 x = make_uint4(__shfl_sync(0xffffffffu, rec.x, from),
                                       __shfl_sync(0xffffffffu, rec.y, from),
                                       __shfl_sync(0xffffffffu, rec.z, from), 0u);
            combine_row<HD>(P, x, w / P.n_head, w % P.n_head, lane);
        }
    }
}

template <int HD, int G, bool SC = false>
int launch_prefill_one(const prefill_params_t<SC>& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                       unsigned ctas, cudaStream_t stream) {
    using C = PCfg<HD, G, SC>;
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
    if (!(configured.load(std::memory_order_acquire) & bit) || bit == 0) {
        cudaError_t e = cudaFuncSetAttribute(slotkv_prefill_tc_kernel<HD, G, SC>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             SC ? C::SMEM_SC : C::SMEM);
        if (e != cudaSuccess) return static_cast<int>(e);
        if constexpr (SC) {
            // the register hand-over assumes 128 registers a thread; with
            // fewer the softmax warps' request could never be met
            cudaFuncAttributes fa;
            e = cudaFuncGetAttributes(&fa, slotkv_prefill_tc_kernel<HD, G, SC>);
            if (e != cudaSuccess) return static_cast<int>(e);
            if (fa.numRegs != 128) return static_cast<int>(cudaErrorInvalidConfiguration);
            // the attention kernel's shared-memory carve-out for the kernels
            // around it, so the SMs need no reconfiguration between them
            const int carve = cudaSharedmemCarveoutMaxShared;
            const cudaFuncAttribute which = cudaFuncAttributePreferredSharedMemoryCarveout;
            if ((e = cudaFuncSetAttribute(slotkv_scored_front_kernel<HD, C::MT, C::BK>, which, carve)) !=
                    cudaSuccess ||
                (e = cudaFuncSetAttribute(slotkv_prefill_prep_kernel<HD, SC>, which, carve)) != cudaSuccess ||
                (e = cudaFuncSetAttribute(slotkv_scored_plan_kernel<C::MT, C::BK, 1024, 1>, which, carve)) !=
                    cudaSuccess ||
                (e = cudaFuncSetAttribute(slotkv_scored_plan_kernel<C::MT, C::BK, 1024, 8>, which, carve)) !=
                    cudaSuccess ||
                (e = cudaFuncSetAttribute(slotkv_combine_kernel<HD>, which, carve)) != cudaSuccess)
                return static_cast<int>(e);
        }
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    uint32_t groups = prep_groups(p.n_head, p.n_kv_head);
    if constexpr (SC)
        if (p.shared.lens) groups = prep_q_groups(p.n_head);
    const uint32_t warps = p.n_tok * groups;
    // the plan (one CTA) first, then prep beside it as its programmatic
    // dependent; the attention kernel waits for both (a plain call's by stream
    // order, a scored call's as a programmatic dependent of prep, whose last
    // CTA ends after the plan).  Prep starts only once the plan runs, hence
    // after the previous call's attention kernel has finished reading the rows
    // and q workspace that prep overwrites.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if constexpr (SC) {
        // Scored calls: a chain of programmatic dependents.  In a shared call
        // the decode plan comes first, and this plan runs beside it (it has
        // waited for the work before the call); otherwise this plan starts
        // the chain, and its launch overlaps the end of the work before.
        if (p.n_tok <= kFrontRows) {
            constexpr uint32_t W = kFrontThreads / 32;
            cfg.gridDim = dim3(1 + (warps + W - 1) / W);
            cfg.blockDim = dim3(kFrontThreads);
            cfg.dynamicSmemBytes = prep_smem_bytes<HD>(W);
            e = cudaLaunchKernelEx(&cfg, slotkv_scored_front_kernel<HD, C::MT, C::BK>, p);
        } else {
            cfg.gridDim = dim3(1);
            cfg.blockDim = dim3(1024);
            auto plan = p.n_tok <= 1024 ? slotkv_scored_plan_kernel<C::MT, C::BK, 1024, 1>
                                        : slotkv_scored_plan_kernel<C::MT, C::BK, 1024, 8>;
            e = cudaLaunchKernelEx(&cfg, plan, p);
        }
        if (e != cudaSuccess) return static_cast<int>(e);
    } else {
        slotkv_prefill_plan_kernel<C::MT><<<1, 1024, 0, stream>>>(p);
    }
    if (!SC || p.n_tok > kFrontRows) {
        cfg.gridDim = dim3((warps + 3) / 4);
        cfg.blockDim = dim3(128);
        cfg.dynamicSmemBytes = prep_smem_bytes<HD>();
        e = cudaLaunchKernelEx(&cfg, slotkv_prefill_prep_kernel<HD, SC>, p);
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    if constexpr (SC) {
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(C::THREADS_SC);
        cfg.dynamicSmemBytes = C::SMEM_SC;
        e = cudaLaunchKernelEx(&cfg, slotkv_prefill_tc_kernel<HD, G, SC>, tmK, tmV, p);
        if (e != cudaSuccess) return static_cast<int>(e);
        if (!p.shared.lens) {  // join the splits, if any
            const uint32_t most = kCombineCtas * p.sms, rows = (p.n_tok * p.n_head + 3) / 4;
            cfg.gridDim = dim3(rows < most ? rows : most);
            cfg.blockDim = dim3(128);
            cfg.dynamicSmemBytes = 0;
            e = cudaLaunchKernelEx(&cfg, slotkv_combine_kernel<HD>, p);
            if (e != cudaSuccess) return static_cast<int>(e);
        }
    } else {
        slotkv_prefill_tc_kernel<HD, G, SC><<<ctas, C::THREADS, C::SMEM, stream>>>(tmK, tmV, p);
    }
    return static_cast<int>(cudaGetLastError());
}

template <int HD, bool SC = false>
int launch_prefill_hd(int G, const prefill_params_t<SC>& p, const CUtensorMap& tmK,
                      const CUtensorMap& tmV, unsigned ctas, cudaStream_t stream) {
    switch (G) {
        case 1: return launch_prefill_one<HD, 1, SC>(p, tmK, tmV, ctas, stream);
        case 2: return launch_prefill_one<HD, 2, SC>(p, tmK, tmV, ctas, stream);
        case 3: return launch_prefill_one<HD, 3, SC>(p, tmK, tmV, ctas, stream);
        case 4: return launch_prefill_one<HD, 4, SC>(p, tmK, tmV, ctas, stream);
        case 5: return launch_prefill_one<HD, 5, SC>(p, tmK, tmV, ctas, stream);
        case 6: return launch_prefill_one<HD, 6, SC>(p, tmK, tmV, ctas, stream);
        case 7: return launch_prefill_one<HD, 7, SC>(p, tmK, tmV, ctas, stream);
        case 8: return launch_prefill_one<HD, 8, SC>(p, tmK, tmV, ctas, stream);
        default: return static_cast<int>(cudaErrorInvalidValue);
    }
}

}  // namespace slotkv
