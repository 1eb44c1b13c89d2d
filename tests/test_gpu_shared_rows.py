"""Shared steps of more rows than a plan takes at once."""
import math

import pytest
import torch

from plain64 import F64, check, norm_rope, row_attention
from sequence_slot_kv_gb300 import Scores, SlotKV
from test_gpu_scored import EPS, Layer, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,G,n_kv,B,plen", [(64, 8, 8, 1130, 96), (128, 4, 2, 1500, 500),
                                              (64, 4, 1, 9001, 130), (64, 8, 8, 2500, 40),
                                              (128, 1, 1, 1025, 2000)])
def test_shared_steps_of_many_rows(hd, G, n_kv, B, plen):
    """More rows than one round of the plan at one row a thread, and more than one
    round at eight; rows without a prefix and of other lengths among them.
    The last ones are few tiles, so split."""
    L = Layer(B, 3, n_kv, G, hd, B, seed=B, sinks=True, slopes=True)
    r = torch.Generator().manual_seed(B)
    n_pre = 5
    PK, PV = L.rnd(n_pre, plen, n_kv, hd), L.rnd(n_pre, plen, n_kv, hd)
    pkv = SlotKV(n_pre, plen, n_kv, hd, 1, L.n_head, k_buf=PK, v_buf=PV)
    psl = sorted(torch.randint(0, n_pre, (B,), generator=r).tolist())
    pl = torch.randint(1, plen + 1, (B,), generator=r).tolist()
    own = torch.randint(0, 3, (B,), generator=r).tolist()
    for b in range(0, B, 97):
        psl[b], pl[b] = n_pre + b, 0
    pl[-1], own[-1] = plen, 2
    slots = torch.randperm(B, generator=r).tolist()
    pos = [a + b for a, b in zip(pl, own)]
    K0, V0 = L.K.clone(), L.V.clone()
    q, k, v = L.step(B)
    out = torch.full((B, L.n_head, hd), math.nan, device="cuda")
    L.kv.decode_batch_attn_shared(q, k, v, i32(pos), i32(slots), pkv, i32(psl), i32(pl),
                                  *L.params(), Scores(15.0, plen - 5, L.slopes), out, EPS, L.scale)
    assert L.kv.get_status() == 0
    position = torch.tensor(pos, device="cuda")
    at = torch.tensor(slots, device="cuda"), torch.tensor(own, device="cuda")
    k64 = norm_rope(k, L.kw, position, L.inv, EPS)
    assert float((L.K[at].to(F64) - k64).abs().max()) <= 2.0 ** -20 * float(k64.abs().max())
    K0[at], V0[at] = L.K[at], v
    assert torch.equal(L.K, K0) and torch.equal(L.V, V0)
    q64 = norm_rope(q, L.qw, position, L.inv, EPS)
    rows = sorted({0, 1, 96, 97, 1023, B - 1, *torch.randint(0, B, (300,), generator=r).tolist()})
    outs, tols = [], []
    for b in rows:
        keys = torch.cat([PK[psl[b] if pl[b] else 0, :pl[b]], L.K[slots[b], :own[b] + 1]])
        vals = torch.cat([PV[psl[b] if pl[b] else 0, :pl[b]], L.V[slots[b], :own[b] + 1]])
        t = torch.arange(pos[b] + 1, device="cuda")
        o, tol = row_attention(q64[b], keys, vals, pos[b], t, t > pos[b] - (plen - 5), L.scale, 15.0,
                               L.slopes, L.sinks)
        outs.append(o)
        tols.append(tol)
    assert bool(torch.isfinite(out).all())
    check(out[rows], outs, tols, "shared")
    L.kv.free()
    pkv.free()
