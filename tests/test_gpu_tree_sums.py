"""What the tensor core's cut sums leave of a tree call's outputs: values that
nothing is cut from come back to the bit, others without a bias."""
import random

import pytest
import torch

from tree64 import Case, tree

pytestmark = pytest.mark.gpu


def alone(hd, how, seed):
    """Rows that attend one key each, their own."""
    n = 40
    if how == "roots":
        return Case([(0, [-1] * n), (0, [-1] * 7)], 2, 3, hd, seed=seed)
    return Case([(200, tree(random.Random(seed), n, 4)), (3, [-1, 0])], 2, 3, hd, seed=seed, window=1)


def ran(c):
    kv = c.handle()
    c.run(kv)
    torch.cuda.synchronize()
    assert kv.get_status() == 0
    kv.free()
    return c.out[:c.rows]


def own_values(c):
    return c.v_new[:c.rows].repeat_interleave(c.G, 1)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("how", ["roots", "window"])
def test_a_row_alone_returns_its_value(hd, how):
    """The weight is 1 and the value fits the 11 bits of a product's high part (it
    came from 16 bits): nothing is cut, so nothing is to be put back."""
    c = alone(hd, how, 1)
    c.v_new.copy_(c.v_new.bfloat16().float())
    c.v_new[0], c.v_new[1], c.v_new[2] = 1.0, -3.0, 2.0 ** -60
    assert torch.equal(ran(c), own_values(c))


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("past", [127, 255, 4095])
def test_a_constant_history_returns_its_value(hd, past):
    """q' = 0, so every weight is 1; 2^k keys with one value of 8 bits: their sum and
    its quotient are exact."""
    c = Case([(past, [-1]), (past, [-1, -1, -1])], 2, 4, hd, seed=3)
    c.qw.zero_()
    value = torch.randn(2, hd, device="cuda").bfloat16().float()
    c.V[:], c.v_new[:] = value, value
    assert torch.equal(ran(c), own_values(c))


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("how", ["roots", "window"])
def test_any_value_alone(hd, how):
    """Of a value's 13 low bits 11 are read: what is cut is below 3 units of its last
    place, what is put back below 2, and the joined sum is rounded once: below 3.5
    units.  On average 7/8 of a unit is cut (bits 0 and 1 of the 13 where bit 12 is
    set, bit 0 where 11 is the highest, with uniform bits 3/4 + 1/8) and as much put
    back: of some 12 thousand values and more, each off by about a unit, the mean is
    0 within 0.05 units."""
    c = alone(hd, how, 2)
    got, want = ran(c).double(), own_values(c).double()
    unit = 2.0 ** (torch.floor(torch.log2(want.abs())) - 23)
    off = (got - want) / unit
    assert float(off.abs().max()) <= 3.5
    assert abs(float((off * want.sign()).mean())) <= 0.05


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("channels", ["first", "last", "both"])
def test_keys_of_few_channels(hd, channels):
    """Half of the keys have their whole product with q in four channels, so their
    sums are cut in another way than those of keys that have it everywhere."""
    c = Case([(1500, tree(random.Random(hd), 20, 4)), (90, tree(random.Random(1), 9, 2))], 2, 4, hd, seed=hd)
    few = torch.zeros(hd, device="cuda")
    if channels in ("first", "both"):
        few[:4] = 1
    if channels in ("last", "both"):
        few[-4:] = 1
    c.K[:, ::2] *= few * (hd / few.sum()).sqrt()
    c.K *= 4.0
    kv = c.handle()
    K0, V0 = c.K.clone(), c.V.clone()
    c.run(kv)
    c.check(K0, V0)
    assert kv.get_status() == 0
    kv.free()
