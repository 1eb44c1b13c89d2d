"""The workspace that scored prefills and shared steps share on a handle: its
size, and calls of other shapes one after another on it."""
import math

import pytest
import torch

from plain64 import check
from sequence_slot_kv_gb300 import Scores, SlotKV
from test_gpu_scored import EPS, Layer, check_cache, i32, want_rows
from test_gpu_shared import shared_want

pytestmark = pytest.mark.gpu


def free_bytes():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


def calls(L, n, PK, pkv):
    """A scored prefill of n tokens and a shared step of two rows, as closures."""
    q, dq = L.step(n), L.step(2)
    out, dout = torch.empty(n, L.n_head, L.hd, device="cuda"), torch.empty(2, L.n_head, L.hd, device="cuda")
    pos, slots = i32(list(range(n))), i32([2] * n)
    dpos, dslots, zero, plen = i32([200, 210]), i32([0, 1]), i32([0, 0]), i32([200, 200])
    return (lambda: L.kv.prefill_batch_attn_scored(*q, pos, slots, *L.params(), None, out, EPS, L.scale),
            lambda: L.kv.decode_batch_attn_shared(*dq, dpos, dslots, pkv, zero, plen, *L.params(), None,
                                                  dout, EPS, L.scale))


@pytest.mark.parametrize("shared_first", [False, True])
def test_size(shared_first):
    """A handle of few rows holds few partial results, and one buffer of them for
    both kinds of call: at 64 splits of 40 rows of 8 heads of 64 floats, 5.4
    MB (allocations come in 2 MB pieces), besides 0.1 MB of q and items."""
    PK = torch.randn(1, 200, 2, 64, device="cuda")
    pkv = SlotKV(1, 200, 2, 64, 1, 8, k_buf=PK, v_buf=PK)
    warm, L = [Layer(3, 64, 2, 4, 64, 40, seed=s) for s in (1, 2)]
    for c in calls(warm, 40, PK, pkv):  # (the kernels are loaded here)
        c()
    order = calls(L, 40, PK, pkv)
    a = free_bytes()
    order[shared_first]()
    b = free_bytes()
    order[not shared_first]()
    c = free_bytes()
    assert a - b <= 12 << 20, f"the first call took {a - b} bytes"
    assert b - c == 0, f"the other kind of call took {b - c} bytes more"
    assert L.kv.get_status() == 0
    for x in (warm.kv, L.kv, pkv):
        x.free()


@pytest.mark.parametrize("hd,max_rows", [(64, 1200), (128, 1200), (64, 30000)])
def test_calls_of_other_shapes_one_after_another(hd, max_rows):
    """Prefills and shared steps of other sizes in turn on one handle, split and
    not, each from a cache and an output that hold nothing of the call before.
    At 30000 rows shared steps have partial results of their own."""
    n_kv, G, ctx, plen = 2, 4, 2300, 700
    L = Layer(5, ctx, n_kv, G, hd, max_rows, seed=hd, sinks=True)
    PK, PV = L.rnd(2, plen, n_kv, hd), L.rnd(2, plen, n_kv, hd)
    pkv = SlotKV(2, plen, n_kv, hd, 1, L.n_head, k_buf=PK, v_buf=PV)
    K0, V0 = L.K.clone(), L.V.clone()
    sc = Scores(cap=11.0)
    for kind, x in (("prefill", (2200, 40)), ("shared", 5), ("prefill", (0, 900)), ("shared", 3),
                    ("shared", 5), ("prefill", (2100, 3)), ("shared", 2)):
        L.K.copy_(K0)
        L.V.copy_(V0)
        if kind == "prefill":
            past, n = x
            pos, slots = list(range(past, past + n)), [1] * n
            q = L.step(n)
            where = list(zip(slots, pos))
            L.V[1, past:past + n] = math.nan
            K64, V64, outs, tols = want_rows(L, *q, pos, where, lambda b, t: (1, t), True, 11.0)
            out = torch.full((n, L.n_head, hd), math.nan, device="cuda")
            L.kv.prefill_batch_attn_scored(*q, i32(pos), i32(slots), *L.params(), sc, out, EPS, L.scale)
        else:
            n, slots = x, [3, 1, 0, 4, 2][:x]
            pl = [plen, plen - 50, plen, 0, 300][:x]
            psl = [0, 0, 0, 9, 1][:x]
            pos = [a + 20 * b for b, a in enumerate(pl)]
            q = L.step(n)
            for s, p, m in zip(slots, pos, pl):
                L.V[s, p - m:] = math.nan
            K64, V64, outs, tols, where = shared_want(L, PK, PV, *q, pos, slots, psl, pl, 11.0)
            out = torch.full((n, L.n_head, hd), math.nan, device="cuda")
            L.kv.decode_batch_attn_shared(*q, i32(pos), i32(slots), pkv, i32(psl), i32(pl),
                                          *L.params(), sc, out, EPS, L.scale)
        assert L.kv.get_status() == 0
        check(out, outs, tols, f"{kind} {x}")
        check_cache(L, K64, V64, where)
    L.kv.free()
    pkv.free()
