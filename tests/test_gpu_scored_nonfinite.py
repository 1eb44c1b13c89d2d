"""V values that are not finite in the tensor-core calls: they reach the rows
that attend them, leave every other row's bits alone, and cost the other
sequences of the call nothing."""
import math

import pytest
import torch

from plain64 import F64, check, norm_rope, row_attention
from sequence_slot_kv_gb300 import Scores, SlotKV
from test_gpu_scored import EPS, Layer, i32

pytestmark = pytest.mark.gpu


def wanted(L, q, pos, slots, rows, K=None, V=None, doc=None, **rule):
    """Outputs and tolerances of the given rows, from the cache as the call left it."""
    K, V = L.K if K is None else K, L.V if V is None else V
    q64 = norm_rope(q, L.qw, torch.tensor(pos, device="cuda"), L.inv, EPS)
    outs, tols = [], []
    for b in rows:
        t = torch.arange(pos[b] + 1, device="cuda")
        o, tol = row_attention(q64[b], K[slots[b], :pos[b] + 1], V[slots[b], :pos[b] + 1], pos[b], t,
                               t >= (doc[b] if doc else 0), L.scale, slopes=L.slopes, sinks=L.sinks,
                               **rule)
        outs.append(o)
        tols.append(tol)
    return outs, tols


def time_of(call, times=5):
    best = math.inf
    for _ in range(times):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("hd,bad", [(64, math.inf), (128, math.nan)])
def test_one_value_beside_long_sequences(hd, bad):
    """Three sequences behind 12000 keys and a short one with one infinity or NaN,
    in a call that is not split: the long ones keep their bits, and the call
    takes as long as without it.  (One bad value costs one look at one tile of
    keys: within a fifth of the call; half as much again is allowed.)"""
    G, n_kv, past = 8, 8, 12000
    mt = 128 // G
    fresh = [13 * mt, 13 * mt, 13 * mt, mt]  # 40 tiles x 8 kv heads
    start = [past, past - 777, past, 3]
    n = sum(fresh)
    L = Layer(4, past + 13 * mt, n_kv, G, hd, n, seed=hd)
    pos = [p for s in range(4) for p in range(start[s], start[s] + fresh[s])]
    slots = [s for s in range(4) for _ in range(fresh[s])]
    q, k, v = L.step(n)
    first = n - mt
    args = [i32(pos), i32(slots), *L.params(), Scores(cap=30.0)]
    outs = [torch.full((n, L.n_head, hd), math.nan, device="cuda") for _ in range(2)]

    def call(out):
        L.kv.prefill_batch_attn_scored(q, k, v, *args, out, EPS, L.scale)

    call(outs[0])
    finite = time_of(lambda: call(outs[0]))
    v[first + 2, 5, 9] = bad
    call(outs[1])
    with_bad = time_of(lambda: call(outs[1]))
    assert L.kv.get_status() == 0
    assert torch.equal(outs[0][:first + 2], outs[1][:first + 2])
    rows = list(range(first, n))
    want, tols = wanted(L, q, pos, slots, rows, cap=30.0)
    assert bool(torch.isfinite(want[1]).all()) and not bool(torch.isfinite(want[2]).all())
    check(outs[1][first:], want, tols, "prefill")
    assert with_bad <= 1.5 * finite, f"{with_bad:.3f} ms with one value not finite, {finite:.3f} without"
    L.kv.free()


@pytest.mark.parametrize("hd", [64, 128])
def test_values_at_both_ends_of_a_long_history(hd):
    """Values in the first and the last tiles of a history of 1024 tiles, and
    documents that begin after none, one or all of them."""
    n_kv, G, n = 8, 1, 39 * 128
    bk = 32 if hd == 128 else 64
    far = 1024 * bk
    ctx = far + n + 200
    L = Layer(1, ctx, n_kv, G, hd, n, seed=hd + 1, sinks=True)
    L.V[0, 5, :, 7] = math.inf
    L.V[0, far + 5, :, 8] = -math.inf
    L.V[0, far + 6, 3, 7] = -math.inf  # the first one's sum becomes NaN
    L.V[0, far - 1, 2, 20] = math.nan
    pos = list(range(ctx - n, ctx))
    doc = [(0, 6, far + 6, far + 7)[b % 4] for b in range(n)]
    q, k, v = L.step(n)
    out = torch.full((n, L.n_head, hd), math.nan, device="cuda")
    L.kv.prefill_batch_attn_scored(q, k, v, i32(pos), i32([0] * n), *L.params(),
                                   Scores(doc_start=i32(doc)), out, EPS, L.scale)
    assert L.kv.get_status() == 0
    rows = [0, 1, 2, 3, 128, 1001, 2002, 3003, n - 4, n - 3, n - 2, n - 1]
    want, tols = wanted(L, q, pos, [0] * n, rows, doc=doc)
    assert bool(torch.isnan(want[0]).any()) and bool(torch.isinf(want[0]).any())
    assert bool(torch.isfinite(want[3]).all())
    check(out[rows], want, tols, "prefill")
    L.kv.free()


@pytest.mark.parametrize("hd", [64, 128])
def test_values_in_a_hundred_places_of_a_long_history(hd):
    """More places, ten tiles apart, than the kernel keeps note of for an item:
    NaN in the first ten, infinities in the others, documents that begin before,
    between and after them."""
    n_kv, G, n = 8, 1, 39 * 128
    apart = 10 * (32 if hd == 128 else 64)
    ctx = 100 * apart + n + 100
    L = Layer(1, ctx, n_kv, G, hd, n, seed=hd + 5)
    keys = [apart * j + j for j in range(100)]
    for j, key in enumerate(keys):
        L.V[0, key, :, j % (32 if j < 60 else 16)] = math.nan if j < 10 else math.inf
    pos = list(range(ctx - n, ctx))
    starts = [0, keys[9], keys[9] + 1, keys[70], keys[99], keys[99] + 1]
    doc = [starts[b % 6] for b in range(n)]
    q, k, v = L.step(n)
    out = torch.full((n, L.n_head, hd), math.nan, device="cuda")
    L.kv.prefill_batch_attn_scored(q, k, v, i32(pos), i32([0] * n), *L.params(),
                                   Scores(doc_start=i32(doc)), out, EPS, L.scale)
    assert L.kv.get_status() == 0
    rows = [*range(6), *range(2004, 2010), *range(n - 6, n)]
    want, tols = wanted(L, q, pos, [0] * n, rows, doc=doc)
    assert [int((~torch.isfinite(w[0])).sum()) for w in want[:6]] == [32, 32, 32, 16, 1, 0]
    assert [int(torch.isnan(w[0]).sum()) for w in want[:6]] == [10, 1, 0, 0, 0, 0]
    check(out[rows], want, tols, "prefill")
    L.kv.free()


@pytest.mark.parametrize("hd,G", [(64, 8), (128, 4), (64, 1)])
def test_every_cta_takes_many_short_items(hd, G):
    """Hundreds of sequences of a few tokens, one key tile each, some with a value
    that is not finite: what one item met does not reach the items after it."""
    n_kv, n_seq, r = 8, 600, torch.Generator().manual_seed(hd + G)
    lens = torch.randint(1, 5, (n_seq,), generator=r).tolist()
    n = sum(lens)
    L = Layer(n_seq, 8, n_kv, G, hd, n, seed=hd * G)
    pos = [p for m in lens for p in range(m)]
    slots = [s for s, m in enumerate(lens) for _ in range(m)]
    q, k, v = L.step(n)
    clean = v.clone()
    values = [math.inf, -math.inf, math.nan]
    hit = [b for b in range(n) if int(torch.randint(0, 4, (1,), generator=r)) == 0]
    for b in hit:
        v[b, int(torch.randint(0, n_kv, (1,), generator=r)), b % hd] = values[b % 3]
    outs = []
    for vv in (clean, v):
        out = torch.full((n, L.n_head, hd), math.nan, device="cuda")
        L.kv.prefill_batch_attn_scored(q, k, vv, i32(pos), i32(slots), *L.params(), None, out, EPS,
                                       L.scale)
        outs.append(out)
    assert L.kv.get_status() == 0
    touched = {slots[b] for b in hit}
    same = torch.tensor([s not in touched for s in slots], device="cuda")
    assert torch.equal(outs[0][same], outs[1][same])
    rows = [b for b in range(n) if slots[b] in touched]
    want, tols = wanted(L, q, pos, slots, rows)
    check(outs[1][rows], want, tols, "prefill")
    L.kv.free()


@pytest.mark.parametrize("hd", [64, 128])
def test_one_value_in_a_prefix(hd):
    """Two prefixes of one shared call, one with an infinity in its first keys;
    too many tiles to be split."""
    G, n_kv, plen = 8, 8, 9000
    mt = 128 // G
    B, own = 40 * mt, 4
    L = Layer(B, own, n_kv, G, hd, B, seed=hd + 2)
    PK, PV = L.rnd(2, plen, n_kv, hd), L.rnd(2, plen, n_kv, hd)
    pkv = SlotKV(2, plen, n_kv, hd, 1, L.n_head, k_buf=PK, v_buf=PV)
    psl = [int(b < mt) for b in range(B)]  # the first tile's rows are on prefix 1
    args = [i32([plen] * B), i32(list(range(B))), pkv, i32(psl), i32([plen] * B), *L.params(), None]
    q, k, v = L.step(B)
    outs = [torch.full((B, L.n_head, hd), math.nan, device="cuda") for _ in range(2)]

    def call(out):
        L.kv.decode_batch_attn_shared(q, k, v, *args, out, EPS, L.scale)

    call(outs[0])
    finite = time_of(lambda: call(outs[0]))
    PV[1, 3, 2, 11] = math.inf
    call(outs[1])
    with_bad = time_of(lambda: call(outs[1]))
    assert L.kv.get_status() == 0
    assert torch.equal(outs[0][mt:], outs[1][mt:])
    q64 = norm_rope(q[:2], L.qw, torch.tensor([plen] * 2, device="cuda"), L.inv, EPS)
    want, tols = [], []
    for b in range(2):
        o, tol = row_attention(q64[b], torch.cat([PK[1], L.K[b, :1]]), torch.cat([PV[1], L.V[b, :1]]),
                               plen, torch.arange(plen + 1, device="cuda"),
                               torch.ones(plen + 1, dtype=torch.bool, device="cuda"), L.scale)
        want.append(o)
        tols.append(tol)
    assert bool(torch.isinf(want[0]).any())
    check(outs[1][:2], want, tols, "shared")
    assert with_bad <= 1.5 * finite, f"{with_bad:.3f} ms with one value not finite, {finite:.3f} without"
    L.kv.free()
    pkv.free()


@pytest.mark.parametrize("hd", [64, 128])
def test_a_value_that_no_row_attends(hd):
    """Between the keys of a tile's first rows and those of its last: no row changes."""
    pos = [*range(3, 11), *range(700, 732)]
    doc = [0] * 8 + [650] * 32
    n = len(pos)
    L = Layer(1, 800, 1, 4, hd, n, seed=hd + 3)
    q, k, v = L.step(n)
    outs = []
    for x in (1.0, math.nan):
        L.V[0, 100:600] = x
        out = torch.full((n, 4, hd), math.nan, device="cuda")
        L.kv.prefill_batch_attn_scored(q, k, v, i32(pos), i32([0] * n), *L.params(),
                                       Scores(doc_start=i32(doc)), out, EPS, L.scale)
        outs.append(out)
    assert L.kv.get_status() == 0 and bool(torch.isfinite(outs[0]).all())
    assert torch.equal(outs[0], outs[1])
    L.kv.free()
