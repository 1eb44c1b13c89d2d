// score_rule.cuh -- the score rule of the scored calls: a tanh cap on the
// scaled scores (soft-capped attention), a bias linear in the distance, and
// masks that limit each row to one range of keys.
//
// Row at position p (a key's position t): s = scale <q', k'>; with a cap c,
// s <- c tanh(s / c); with slopes, s <- s - slope_h |p - t|; the row attends
// t iff lo <= t <= hi, where lo = max(doc_start, p + 1 - window) and hi = p,
// or in a prefill max(p, prefix_end - 1).  Scores are kept in base 2 (times
// log2 e), so the cap's two constants and the slopes carry that factor.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "params.h"

namespace slotkv {

constexpr float kRuleLog2e = 1.4426950408889634f;

// tanh for the cap, with a few ulp of relative error everywhere.  Above 5/8
// it is (1 - e) / (1 + e) with e = exp(-2 |y|) <= 0.29 (1 - e loses nothing
// there); below, Lambert's continued fraction y / (1 + y^2 / (3 + y^2 / (5 +
// ...))) cut after the 9, whose error at 5/8 is below 2^-27 relative.  One
// division serves both: numerator and denominator are selected first.
// NaN takes the first form and stays NaN; +-inf gives +-1.
__device__ __forceinline__ float cap_tanh(float y) {
    const float a = fabsf(y), y2 = y * y;
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * (-2.f * kRuleLog2e)));
    const bool small = a < 0.625f;
    const float num = small ? a * fmaf(y2, y2 + 105.f, 945.f) : 1.f - e;
    const float den = small ? fmaf(y2, fmaf(y2, 15.f, 420.f), 945.f) : 1.f + e;
    return copysignf(__fdividef(num, den), y);
}

// Cap N scores of one thread, all 32 lanes of the warp together.  The
// tensor-core prefill's softmax has little time for it and cap_tanh is some
// twenty instructions, so scores well inside the cap -- the usual case: caps
// are several times the scores -- take the Taylor series tanh(y) / y = 1 -
// u / 3 + 2 u^2 / 15 - 17 u^3 / 315, u = y^2, two scores per instruction and
// the cap's constant folded into the coefficients; for |y| <= 1/8 the first
// term left out is below 2^-29.  (cap_in cap_out = 1, so cap_out tanh(y) = s
// tanh(y) / y.)  One score outside sends the warp's part of the tile to
// cap_tanh.  (Caps are 1e-6 .. 1e6: nothing here overflows.)
struct CapSeries {
    float c1, c2, c3;
};
__device__ __forceinline__ CapSeries cap_series(float cap_in) {
    const float k = cap_in * cap_in;
    return {k * (-1.f / 3.f), k * k * (2.f / 15.f), k * k * k * (-17.f / 315.f)};
}
template <int N>
__device__ __forceinline__ void cap_scores(float (&s)[N], const ScoreRule& r, const CapSeries& k) {
    float t4[4] = {0.f, 0.f, 0.f, 0.f};  // four short chains
#pragma unroll
    for (int c = 0; c < N; ++c) t4[c & 3] = fmaxf(t4[c & 3], fabsf(s[c]));
    const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
    if (__any_sync(0xffffffffu, top * r.cap_in > 0.125f)) {
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = r.cap_out * cap_tanh(s[c] * r.cap_in);
        return;
    }
    auto both = [](float x) { return make_float2(x, x); };
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 x = make_float2(s[c], s[c + 1]);
        const float2 u = __fmul2_rn(x, x);
        float2 t = __ffma2_rn(u, both(k.c3), both(k.c2));
        t = __ffma2_rn(u, t, both(k.c1));
        t = __ffma2_rn(u, t, both(1.f));
        const float2 y = __fmul2_rn(x, t);
        s[c] = y.x;
        s[c + 1] = y.y;
    }
}

// One score after cap and bias; slope2 = slope_h log2 e (0: no bias), d = p - t.
__device__ __forceinline__ float apply_rule(float s, float cap_in, float cap_out, float slope2,
                                            bool bias, int d) {
    if (cap_out != 0.f) s = cap_out * cap_tanh(s * cap_in);
    if (bias) s = fmaf(-slope2, fabsf(static_cast<float>(d)), s);
    return s;
}

// First key of a row at position p by its document and the window.
__device__ __forceinline__ uint32_t rule_first(const ScoreRule& r, uint32_t b, uint32_t p) {
    uint32_t lo = r.doc_start ? __ldg(r.doc_start + b) : 0u;
    if (r.window && p >= r.window) {
        const uint32_t w = p - r.window + 1u;
        lo = lo > w ? lo : w;
    }
    return lo;
}

// A row of a scored decode call, in its own slot's positions: p of the new
// key, lo the first key attended (past p: none), len its prefix length.
// ok is false for a row out of range, which every kernel of the call skips:
// a position below its prefix or past its slot, a prefix past its handle's
// slots, a prefix_end past the slot.
struct ScoredRow {
    uint32_t p, lo, hi, len;
    bool ok;
};
__device__ __forceinline__ ScoredRow scored_row(const ScoreRule& rule, const SharedRows& sh,
                                                uint32_t b, uint32_t pos, uint64_t cap,
                                                bool slot_ok, bool prefill) {
    // (every load first: they are in flight together)
    const uint32_t len = sh.lens ? __ldg(sh.lens + b) : 0u;
    const uint32_t pslot = sh.lens ? __ldg(sh.slots + b) : 0u;
    const uint32_t first = rule_first(rule, b, pos);
    const uint32_t end = prefill && rule.prefix_end ? __ldg(rule.prefix_end + b) : 0u;
    ScoredRow r;
    r.len = len;
    r.ok = slot_ok && pos >= len && (len == 0u || (len <= sh.slot_ctx && pslot < sh.n_slots));
    r.p = r.ok ? pos - len : 0u;
    r.ok = r.ok && static_cast<uint64_t>(r.p) < cap && static_cast<uint64_t>(end) <= cap;
    r.lo = first > len ? first - len : 0u;
    r.hi = end > r.p + 1u ? end - 1u : r.p;
    return r;
}

// A row's keys start at the tile holding its first key (its last, when the
// mask leaves none).
__device__ __forceinline__ uint32_t row_base(uint32_t lo, uint32_t hi, uint32_t tile) {
    return (lo < hi ? lo : hi) / tile * tile;
}

}  // namespace slotkv
