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
    ScoredRow r;
    r.len = sh.lens ? __ldg(sh.lens + b) : 0u;
    r.ok = slot_ok && pos >= r.len;
    if (sh.lens && r.len)
        r.ok = r.ok && r.len <= sh.slot_ctx && __ldg(sh.slots + b) < sh.n_slots;
    r.p = r.ok ? pos - r.len : 0u;
    r.ok = r.ok && static_cast<uint64_t>(r.p) < cap;
    const uint32_t first = rule_first(rule, b, pos);
    r.lo = first > r.len ? first - r.len : 0u;
    r.hi = r.p;
    if (prefill && rule.prefix_end) {
        const uint32_t e = __ldg(rule.prefix_end + b);
        if (e > cap) r.ok = false;
        if (e > r.p + 1u) r.hi = e - 1u;
    }
    return r;
}

// A row's keys start at the tile holding its first key (its last, when the
// mask leaves none).
__device__ __forceinline__ uint32_t row_base(uint32_t lo, uint32_t hi, uint32_t tile) {
    return (lo < hi ? lo : hi) / tile * tile;
}

}  // namespace slotkv
