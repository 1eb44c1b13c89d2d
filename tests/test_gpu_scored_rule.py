"""A score rule whose arrays are replaced between calls, both ways the binding
makes a call."""
import math

import pytest
import torch

import sequence_slot_kv_gb300 as skv
from plain64 import F64, check
from sequence_slot_kv_gb300 import Scores
from test_gpu_scored import EPS, Layer, check_cache, i32, want_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("compiled", [True, False])
def test_a_rule_whose_arrays_are_replaced(compiled, monkeypatch):
    """What is assigned to a rule is what the next call uses; what was there
    before is not."""
    if not compiled:
        monkeypatch.setattr(skv, "_call", False)
    L = Layer(4, 96, 2, 2, 64, 4, seed=44, slopes=True)
    pos, slots = [40, 90, 17], [3, 0, 1]
    q = L.step(3)
    K64, V64, _, _ = want_rows(L, *q, pos, list(zip(slots, pos)), lambda b, t: (slots[b], t), False)
    sc, slopes = Scores(9.0, 80, L.slopes, i32([0, 0, 0])), L.slopes
    for doc, factor in (([0, 0, 0], 1.0), ([30, 85, 17], 1.0), (None, 3.0), ([5, 6, 7], None)):
        sc.doc_start = None if doc is None else i32(doc)
        sc.slopes = L.slopes = None if factor is None else slopes * factor
        _, _, outs, tols = want_rows(L, *q, pos, list(zip(slots, pos)), lambda b, t: (slots[b], t),
                                     False, 9.0, 80, doc)
        out = torch.full((3, 4, 64), math.nan, device="cuda")
        L.kv.decode_batch_attn_scored(*q, i32(pos), i32(slots), *L.params(), sc, out, EPS, L.scale)
        check(out, outs, tols, f"documents from {doc}, slopes times {factor}")
    sc.doc_start, sc.slopes, sc.prefix_end = None, None, i32([0, 0, 60])
    _, _, outs, tols = want_rows(L, *q, pos, list(zip(slots, pos)), lambda b, t: (slots[b], t), True,
                                 9.0, 80, None, [0, 0, 60])
    L.kv.prefill_batch_attn_scored(*q, i32(pos), i32(slots), *L.params(), sc, out, EPS, L.scale)
    check(out, outs, tols, "prefix")
    check_cache(L, K64, V64, list(zip(slots, pos)))
    assert L.kv.get_status() == 0
    L.kv.free()


@pytest.mark.parametrize("compiled", [True, False])
def test_a_replaced_array_is_checked(compiled, monkeypatch):
    if not compiled:
        monkeypatch.setattr(skv, "_call", False)
    L = Layer(4, 96, 2, 2, 64, 4, seed=45)
    q, out = L.step(3), torch.full((3, 4, 64), 7.0, device="cuda")
    for name, bad, err in (("doc_start", torch.zeros(3, dtype=torch.int32), ValueError),
                           ("doc_start", i32([0, 0]), ValueError),
                           ("doc_start", i32([0] * 6)[::2], ValueError),
                           ("doc_start", i32([0, 0, 0]).long(), TypeError),
                           ("doc_start", [0, 0, 0], TypeError),
                           ("slopes", torch.zeros(4), ValueError),
                           ("slopes", torch.zeros(4, dtype=F64, device="cuda"), TypeError)):
        sc = Scores(9.0)
        setattr(sc, name, bad)
        with pytest.raises(err, match=name):
            L.kv.decode_batch_attn_scored(*q, i32([1, 2, 3]), i32([0, 1, 2]), *L.params(), sc, out,
                                          EPS, L.scale)
    assert bool((out == 7.0).all()) and L.kv.get_status() == 0
    L.kv.free()
