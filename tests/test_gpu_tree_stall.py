"""What a tree call that ends by a wait that ran out has written."""
import random

import pytest
import torch

import sequence_slot_kv_gb300 as skv
from tree64 import Case, tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("past", [300, 30000])
@pytest.mark.parametrize("first", [True, False])
def test_a_stalled_call_leaves_out_alone(hd, past, first):
    """Every CTA of the attention gives up at its first tile: no row of out is
    written, joined from an earlier call's partial results (past 30000: the rows
    lie in several CTAs) or from a workspace that no call has filled."""
    r = random.Random(hd)
    c = Case([(past, tree(r, 16, 4)), (64, tree(r, 7, 4))], 1, 4, hd, seed=hd)
    kv = c.handle()
    if not first:
        c.run(kv)
        assert kv.get_status() == 0
    c.out.fill_(7.5)
    kv.set_options(skv.OPT_TEST_STALL)
    c.run(kv)
    assert kv.get_status() == skv.DEV_TIMEOUT
    assert bool((c.out == 7.5).all())
    kv.set_options(0)
    K0, V0 = c.K.clone(), c.V.clone()
    c.run(kv)
    c.check(K0, V0)
    assert kv.get_status() == 0
    kv.free()
