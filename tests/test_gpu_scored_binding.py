"""The two ways the binding makes the scored, shared and request-length calls
(compiled, and through ctypes where that is not built): every one of them, one
good call each way."""
import math

import pytest
import torch

import sequence_slot_kv_gb300 as skv
from plain64 import check
from sequence_slot_kv_gb300 import Scores, SlotKV
from test_gpu_scored import EPS, Layer, check_cache, i32, want_rows
from test_gpu_shared import shared_want

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["compiled", "ctypes"])
def way(request, monkeypatch):
    """One way only: a call that would take the other fails."""
    if request.param == "compiled":
        assert skv._compiled(), "the compiled calls are not built"

        def declined(*a, **k):
            raise AssertionError("the compiled call declined good arguments")

        monkeypatch.setattr(skv, "_step_addrs", declined)
        monkeypatch.setattr(skv, "_int_addr", declined)
    else:
        monkeypatch.setattr(skv, "_call", False)
    return request.param


def test_decode_and_prefill(way):
    for name, prefill in (("decode_batch_attn_scored", False), ("prefill_batch_attn_scored", True)):
        L = Layer(5, 96, 2, 3, 64, 6, seed=41, sinks=True, slopes=True)
        pos, slots, doc, pend = [5, 90, 17, 18], [3, 0, 1, 1], [2, 80, 3, 0], [0, 0, 30, 30]
        if not prefill:
            slots, pend = [3, 0, 1, 2], None
        q = L.step(4)
        K64, V64, outs, tols = want_rows(L, *q, pos, list(zip(slots, pos)), lambda b, t: (slots[b], t),
                                         prefill, 7.0, 60, doc, pend)
        out = torch.full((4, 6, 64), math.nan, device="cuda")
        sc = Scores(7.0, 60, L.slopes, i32(doc), i32(pend) if pend else None)
        assert getattr(L.kv, name)(*q, i32(pos), i32(slots), *L.params(), sc, out, EPS, L.scale) is out
        assert L.kv.get_status() == 0
        check(out, outs, tols, name)
        check_cache(L, K64, V64, list(zip(slots, pos)))
        L.kv.free()


def test_paged(way):
    L = Layer(7, 64, 1, 4, 64, 3, seed=42, sinks=True, slopes=True)
    tab, pos, doc = [[6, 1, 0], [2, 5, -1]], [130, 70], [3, 69]
    q = L.step(2)
    where = [(tab[b][p // 64], p % 64) for b, p in enumerate(pos)]
    at = torch.tensor(tab, device="cuda")
    K64, V64, outs, tols = want_rows(L, *q, pos, where, lambda b, t: (at[b, t // 64], t % 64), False,
                                     5.0, 100, doc)
    out = torch.full((2, 4, 64), math.nan, device="cuda")
    L.kv.decode_batch_attn_paged_scored(*q, i32(pos), i32(tab), *L.params(),
                                        Scores(5.0, 100, L.slopes, i32(doc)), out, EPS, L.scale)
    assert L.kv.get_status() == 0
    check(out, outs, tols, "paged")
    check_cache(L, K64, V64, where)
    L.kv.free()


def test_shared(way):
    L = Layer(6, 40, 2, 2, 64, 4, seed=43, sinks=True, slopes=True)
    PK, PV = L.rnd(3, 90, 2, 64), L.rnd(3, 90, 2, 64)
    pkv = SlotKV(3, 90, 2, 64, 1, 4, k_buf=PK, v_buf=PV)
    slots, psl, plen, pos, doc = [5, 0, 2], [1, 2, 2], [90, 33, 0], [100, 60, 39], [4, 35, 0]
    q = L.step(3)
    K64, V64, outs, tols, where = shared_want(L, PK, PV, *q, pos, slots, psl, plen, 6.0, 95, doc)
    out = torch.full((3, 4, 64), math.nan, device="cuda")
    L.kv.decode_batch_attn_shared(*q, i32(pos), i32(slots), pkv, i32(psl), i32(plen), *L.params(),
                                  Scores(6.0, 95, L.slopes, i32(doc)), out, EPS, L.scale)
    assert L.kv.get_status() == 0
    check(out, outs, tols, "shared")
    check_cache(L, K64, V64, where)
    L.kv.free()
    pkv.free()


def test_request_lengths(way):
    kv = SlotKV(9, 64, 1, 64, 1, 1)
    slots, past, fresh = i32([7, 2, 5]), i32([60, 0, 3]), i32([4, 2, 0])
    starts, ts, tp = i32([9] * 4), i32([9] * 7), i32([9] * 7)
    kv.token_map(slots, past, fresh, starts, ts, tp)
    assert starts.tolist() == [0, 4, 6, 6]
    assert ts.tolist() == [7, 7, 7, 7, 2, 2, 9] and tp.tolist() == [60, 61, 62, 63, 0, 1, 9]
    tab = i32([[1, -1, -1], [-1, -1, -1], [4, -1, -1]])
    free, head, after = i32([0, 3, 8, 6, 5, 7]), i32([1]), i32([0])
    kv.extend_tables(i32([64, 0, 3]), i32([65, 1, 1]), tab, free, head, after)
    assert tab.tolist() == [[1, 3, 8], [6, -1, -1], [4, -1, -1]]
    assert head.tolist() == [1] and after.tolist() == [4]
    kv.extend_tables(i32([128]), i32([1]), tab[2:], free, after)
    assert tab[2].tolist() == [4, -1, 5] and after.tolist() == [5]
    assert kv.get_status() == 0
    kv.free()
