"""The score rule object of the Python binding, without a GPU: what is assigned
to its arrays is what a call sees and checks."""
import pytest
import torch

import sequence_slot_kv_gb300 as skv


def test_assigned_arrays_are_the_rules():
    sc = skv.Scores(2.0, 9)
    for name in ("slopes", "doc_start", "prefix_end"):
        t = torch.zeros(3)
        setattr(sc, name, t)
        assert getattr(sc, name) is t and any(x is t for x in sc._args)
        setattr(sc, name, None)
        assert getattr(sc, name) is None
    assert sc._args == (2.0, 9, None, None, None)


@pytest.mark.parametrize("name,t,err", [
    ("doc_start", torch.zeros(3, dtype=torch.int32), ValueError),  # not on the GPU
    ("slopes", torch.zeros(8), ValueError),
    ("slopes", torch.zeros(8, dtype=torch.float64), TypeError),
    ("prefix_end", torch.zeros(3), TypeError),
    ("prefix_end", [0, 0, 0], TypeError)])
def test_assigned_arrays_are_checked_by_the_call(name, t, err):
    sc = skv.Scores(2.0)
    setattr(sc, name, t)
    with pytest.raises(err, match=name):
        skv._scores(sc, 3, 8, 0)


@pytest.mark.parametrize("name", ["cap", "window"])
def test_numbers_are_fixed(name):
    sc = skv.Scores(2.0, 9)
    with pytest.raises(AttributeError):
        setattr(sc, name, 3)
