"""The scored and shared calls under the handle's norm options (weightless V
norm, norm weights as 1 + w), against their definition in 64 bits."""
import copy
import math

import pytest
import torch

import sequence_slot_kv_gb300 as skv
from plain64 import F64, check
from sequence_slot_kv_gb300 import Scores, SlotKV
from test_gpu_scored import EPS, Layer, i32, want_rows
from test_gpu_shared import shared_want

pytestmark = pytest.mark.gpu


def under(L, flags):
    """The layer as the definition sees it under these options."""
    x = copy.copy(L)
    if flags & skv.OPT_NORM_PLUS_ONE:
        x.qw, x.kw = L.qw.to(F64) + 1, L.kw.to(F64) + 1
    return x


def v_of(v, flags):
    v = v.to(F64)
    return v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt() if flags & skv.OPT_VNORM else v


def check_all(L, out, K64, V64, outs, tols, where, what):
    """out, and the new rows of K and V: V's norm is off by a few roundings of
    32 bits (2^-21 relative), which out, an average of V, takes over."""
    vmax = float(V64.abs().max())
    check(out, outs, [t + 2.0 ** -21 * vmax for t in tols], what)
    for name, got, want in (("K", L.K, K64), ("V", L.V, V64)):
        for x, y in where:
            err = float((got[x, y].to(F64) - want[x, y]).abs().max())
            assert err <= 2.0 ** -20 * float(want[x, y].abs().max()), f"{what}: {name}"


@pytest.mark.parametrize("flags", [1, 2, 3])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_norm_options(hd, flags):
    L = Layer(7, 256, 2, 3, hd, 64, seed=hd + flags, sinks=True, slopes=True)
    L.kv.set_options(flags)
    W = under(L, flags)
    # decode over slots
    pos, slots = [3, 255, 100, 64], [1, 0, 5, 2]
    q, k, v = L.step(4)
    sc = Scores(9.0, 90, L.slopes)
    where = list(zip(slots, pos))
    want = want_rows(W, q, k, v_of(v, flags), pos, where, lambda b, t: (slots[b], t), False, 9.0, 90)
    out = torch.full((4, 6, hd), math.nan, device="cuda")
    L.kv.decode_batch_attn_scored(q, k, v, i32(pos), i32(slots), *L.params(), sc, out, EPS, L.scale)
    check_all(L, out, *want, where, "decode")
    # prefill: 40 tokens of slot 3 from position 30
    pos = list(range(30, 70))
    where = [(3, p) for p in pos]
    q, k, v = L.step(40)
    want = want_rows(W, q, k, v_of(v, flags), pos, where, lambda b, t: (3, t), True, 9.0, 90)
    out = torch.full((40, 6, hd), math.nan, device="cuda")
    L.kv.prefill_batch_attn_scored(q, k, v, i32(pos), i32([3] * 40), *L.params(), sc, out, EPS,
                                   L.scale)
    check_all(L, out, *want, where, "prefill")
    # a shared step on a prefix
    if hd < 256:
        PK, PV = L.rnd(1, 300, 2, hd), L.rnd(1, 300, 2, hd)
        pkv = SlotKV(1, 300, 2, hd, 1, 6, k_buf=PK, v_buf=PV)
        slots, psl, plen, own = [4, 6, 0], [0] * 3, [300, 299, 0], [7, 0, 200]
        pos = [a + b for a, b in zip(plen, own)]
        q, k, v = L.step(3)
        *want, where = shared_want(W, PK, PV, q, k, v_of(v, flags), pos, slots, psl, plen, 9.0, 90)
        out = torch.full((3, 6, hd), math.nan, device="cuda")
        L.kv.decode_batch_attn_shared(q, k, v, i32(pos), i32(slots), pkv, i32(psl), i32(plen),
                                      *L.params(), sc, out, EPS, L.scale)
        check_all(L, out, *want, where, "shared")
        pkv.free()
    # decode over the same buffers as a pool of blocks
    pool = SlotKV(7, 256, 2, hd, 4, 6, k_buf=L.K, v_buf=L.V)
    pool.set_options(flags)
    tab = [[4, 1], [2, -1]]
    pos = [300, 17]
    where = [(1, 44), (2, 17)]
    q, k, v = L.step(2)
    want = want_rows(W, q, k, v_of(v, flags), pos, where,
                     lambda b, t: (torch.tensor(tab[b], device="cuda")[t // 256], t % 256), False,
                     9.0, 90)
    out = torch.full((2, 6, hd), math.nan, device="cuda")
    pool.decode_batch_attn_paged_scored(q, k, v, i32(pos), i32(tab), *L.params(), sc, out, EPS,
                                        L.scale)
    check_all(L, out, *want, where, "paged")
    assert L.kv.get_status() == 0 and pool.get_status() == 0
    pool.free()
    L.kv.free()
