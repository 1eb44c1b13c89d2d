"""The scored and shared calls in 64 bits, row by row, from their definition
(include/slotkv.h, slotkv_scores), with the error a 32-bit evaluation may
have.  Plain torch on whatever device the inputs are on."""
import math

import torch

F64 = torch.float64


def norm_rope(x, w, pos, inv_freq, eps, plus_one=False):
    """RoPE at pos of RMSnorm(x) * w; x [rows, heads, hd].  The angle is the f32
    product of position and frequency, by definition."""
    x = x.to(F64)
    x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    x = x * (w.to(F64) + (1.0 if plus_one else 0.0))
    ang = (pos.float()[:, None] * inv_freq[None, :]).to(F64)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def row_attention(q, K, V, p, t, keep, scale, cap=0.0, slopes=None, sinks=None):
    """One row's heads: q [n_head, hd], K and V [keys, n_kv, hd] at positions t,
    keep [keys].  Returns (out [n_head, hd], tol): tol bounds the error of a
    32-bit evaluation.  Masked keys are left out before any arithmetic.

    The bound.  A product of the score is formed to 2^-20 relative (three TF32
    products drop at most that; f32 FMAs less), so a score's error is at most
    2^-20 S with S = scale sum |q_i k_i|, plus 4 ulp (2^-22) of the capped score and of the bias, plus the
    error of q' and k' themselves (a few ulp each: 2^-21 S).  With every score
    off by at most d, each softmax weight is off by a factor within e^(+-2 d),
    and out, an average of V under the weights, by at most 2 d max|V|; the
    weighted sums add 2^-19 max|V| (their own products and a rounding per
    64 keys)."""
    n_head, hd = q.shape
    n_kv = K.shape[1]
    if not bool(keep.any()):
        return torch.zeros(n_head, hd, dtype=F64, device=q.device), 0.0
    K, V, t = K[keep].to(F64), V[keep].to(F64), t[keep]
    qg = q.view(n_kv, -1, hd)
    s = torch.einsum("ngd,tnd->ngt", qg, K) * scale
    S = torch.einsum("ngd,tnd->ngt", qg.abs(), K.abs()).max() * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    d = S * (2.0 ** -20 + 2.0 ** -21) + s.abs().max() * 2.0 ** -22
    if slopes is not None:
        bias = slopes.to(F64).view(n_kv, -1, 1) * (p - t).abs()
        s = s - bias
        # only biases near the row's best score matter: weights further than
        # 2^-40 below it are nothing at either precision
        near = s > s.amax(-1, keepdim=True) - 28.0
        d = d + (bias * near).max() * 2.0 ** -22
    m = s.amax(-1, keepdim=True)
    if sinks is not None:
        sk = sinks.to(F64).view(n_kv, -1, 1)
        m = torch.maximum(m, sk)
    e = torch.exp(s - m)
    den = e.sum(-1, keepdim=True)
    if sinks is not None:
        den = den + torch.exp(sk - m)
    # (an infinite or NaN value reaches every head of its kv head)
    out = torch.einsum("ngt,tnd->ngd", e, V) / den
    vmax = torch.where(torch.isfinite(V), V.abs(), torch.zeros_like(V)).max()
    return out.reshape(n_head, hd), float(vmax * (2 * d + 2.0 ** -19))


def key_range(p, b, prefill, window=0, doc_start=None, prefix_end=None):
    lo = int(doc_start[b]) if doc_start is not None else 0
    if window:
        lo = max(lo, p + 1 - window)
    hi = p
    if prefill and prefix_end is not None:
        hi = max(p, int(prefix_end[b]) - 1)
    return lo, hi


def check(got, want, tols, what):
    """Row by row: |got - want| <= tol of the row; where want is not finite got
    has to be the same."""
    for b, tol in enumerate(tols):
        g, w = got[b].to(F64), want[b]
        fine = torch.isfinite(w)
        assert torch.equal(torch.isnan(g), torch.isnan(w)), f"{what}: NaN places, row {b}"
        assert torch.equal(g[~fine & ~torch.isnan(w)], w[~fine & ~torch.isnan(w)]), f"{what}: row {b}"
        err = float((g - w)[fine].abs().max()) if bool(fine.any()) else 0.0
        assert math.isfinite(err) and err <= tol + 1e-30, f"{what}: row {b} off by {err:.3g} > {tol:.3g}"
