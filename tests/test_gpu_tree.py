"""tree_batch_attn and tree_batch_attn_paged against their definition in 64 bits."""
import random

import pytest
import torch

import sequence_slot_kv_gb300 as skv
from sequence_slot_kv_gb300 import SlotKV
from tree64 import Case, i32, tree

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def go(c, **kw):
    kv = c.handle()
    K0, V0 = c.K.clone(), c.V.clone()
    c.run(kv)
    c.check(K0, V0, **kw)
    assert kv.get_status() == 0
    kv.free()


def requests(seed, lens, width=4):
    r = random.Random(seed)
    return [(past, tree(r, n, width)) for past, n in lens]


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_heads(hd, G):
    lens = [(300, 9), (0, 5), (127, 1), (1, 20), (513, 3)]
    go(Case(requests(G, lens), 2, G, hd, seed=G * hd, sinks=G % 2 == 0, pad=G % 3))


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("past", [0, 1, 63, 64, 127, 128, 129, 255, 256, 2049])
def test_lengths(hd, past):
    """Histories and trees that end on, before and behind multiples of 128."""
    lens = [(past, n) for n in (1, 2, 17, 33)] + [(past, max(1, 128 - past % 128))]
    go(Case(requests(past, lens), 1, 4, hd, seed=past + hd))


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("shape", ["chain", "star", "forest", "binary", "random"])
@pytest.mark.parametrize("n", [33, 256])
def test_shapes(hd, shape, n):
    r = random.Random(n)
    par = {"chain": list(range(-1, n - 1)), "star": [-1] + [0] * (n - 1), "forest": [-1] * n,
           "binary": [(i - 1) // 2 if i else -1 for i in range(n)], "random": tree(r, n, n, 3)}[shape]
    go(Case([(70, par), (130, par[:n // 2])], 1, 2 if hd == 256 else 3, hd, seed=n + hd, sinks=True))


@pytest.mark.parametrize("hd,block", [(64, 64), (64, 128), (64, 192), (128, 32), (128, 96),
                                      (128, 128), (256, 16), (256, 48), (256, 64), (256, 512)])
def test_paged(hd, block):
    lens = [(5 * block - 3, 7), (block, 2 * block % 250 + 1), (0, 3), (777, 31), (block - 1, 1)]
    go(Case(requests(block, lens), 2, 4, hd, block=block, seed=block + hd, sinks=True, pad=2))


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("rule", ["cap", "window", "window1", "slopes", "docs", "all"])
@pytest.mark.parametrize("block", [0, 64])
def test_rules(hd, rule, block):
    lens = [(700, 40), (0, 6), (129, 64), (3, 12), (260, 1)]
    kw = {"cap": dict(cap=4.0), "window": dict(window=100), "window1": dict(window=1),
          "slopes": dict(slopes=True), "docs": dict(docs=[650, 2, 0, 14, 260]),
          "all": dict(cap=2.5, window=37, slopes=True, docs=[690, 0, 131, 2, 1])}[rule]
    go(Case(requests(7, lens, 2), 2, 3, hd, block=block, seed=hd, sinks=rule == "all", **kw))


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_mask_leaves_nothing(hd):
    """Documents that begin behind some or all of the nodes: those rows are zeros."""
    lens = [(200, 9), (40, 3), (0, 5)]
    c = Case([(p, list(range(-1, n - 1))) for p, n in lens], 2, 2, hd, docs=[204, 60, 1000])
    go(c)
    assert float(c.out[:4].abs().max()) == 0 and float(c.out[9:].abs().max()) == 0
    go(Case([(p, list(range(-1, n - 1))) for p, n in lens], 2, 2, hd, docs=[204, 60, 1000], sinks=True))


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("block", [0, 64])
def test_rest_of_the_cache_may_hold_anything(hd, block):
    """Keys behind a request's nodes, blocks of others, rows before a window or a
    document: NaN and infinities there change nothing."""
    lens = [(300, 11), (129, 2), (64, 1)]
    c = Case(requests(3, lens), 2, 4, hd, block=block, window=80, docs=[250, 0, 64], seed=5)
    bad = torch.tensor([NAN, INF, -INF], device="cuda").repeat(c.K.numel())[:c.K.numel()].view(c.K.shape)
    K, V = bad.clone(), bad.flip(0).clone()
    for r, (past, par) in enumerate(c.reqs):
        lo = max(c.docs[r], past + 1 - 80, 0)
        at = c.at(r, torch.arange(lo, past, device="cuda"))
        K[at], V[at] = c.K[at], c.V[at]
    c.K, c.V = K, V
    go(c)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_branches_do_not_touch_each_other(hd, value):
    """A node whose value or key is not finite reaches itself and its descendants."""
    par = [-1, 0, 0, 1, 1, 2, 2, 3, 5]
    for where in ("v", "k", "q"):
        c = Case([(150, par), (20, par)], 2, 4, hd, seed=hd)
        {"v": c.v_new, "k": c.k_new, "q": c.q}[where][1, 0, 3] = value
        if where == "v":
            go(c)
            continue
        kv = c.handle()
        K0, V0 = c.K.clone(), c.V.clone()
        clean = Case([(150, par), (20, par)], 2, 4, hd, seed=hd)
        clean.run(kv2 := clean.handle())
        c.run(kv)
        hit, heads = ([1, 3, 4, 7], 4) if where == "k" else ([1], 1)
        rest = [i for i in range(18) if i not in hit]
        assert torch.equal(c.out[rest], clean.out[rest])
        assert bool(torch.isnan(c.out[hit, :heads]).all())
        assert torch.equal(c.out[hit, heads:], clean.out[hit, heads:])
        kv.free(), kv2.free()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("where", [0, 77, 128, 299])
def test_history_values_not_finite(hd, where):
    c = Case(requests(1, [(300, 8), (300, 70)]), 2, 3, hd, window=230, seed=2)
    at = c.at(0, i32([where]).long())
    c.V[at[0], at[1], 1, 5] = INF
    c.V[at[0], at[1], 0, 2] = NAN
    at = c.at(1, i32([where]).long())
    c.V[at[0], at[1], 0, 0] = -INF
    c.V[at[0], at[1], 0, 1] = INF
    go(c)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_options(hd):
    for flags in (skv.OPT_VNORM, skv.OPT_NORM_PLUS_ONE, skv.OPT_VNORM | skv.OPT_NORM_PLUS_ONE):
        c = Case(requests(1, [(200, 12), (5, 3)]), 2, 2, hd, seed=flags)
        kv = c.handle()
        kv.set_options(flags)
        K0, V0 = c.K.clone(), c.V.clone()
        c.run(kv)
        c.check(K0, V0, vnorm=bool(flags & skv.OPT_VNORM),
                plus_one=bool(flags & skv.OPT_NORM_PLUS_ONE))
        kv.free()


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_plain_rule_is_none(hd):
    c = Case(requests(4, [(333, 21)]), 2, 2, hd)
    kv = c.handle()
    a = c.run(kv).clone()
    assert torch.equal(c.run(kv, scores=None), a)
    kv.free()


def test_chain_is_a_prefill():
    """A chain attends what a causal prefill of the same tokens attends."""
    for hd in (64, 128, 256):
        c = Case([(100, list(range(-1, 29)))], 2, 4, hd, seed=9)
        kv = c.handle()
        a = c.run(kv).clone()
        K, V = c.K.clone(), c.V.clone()
        n = c.rows
        out = torch.empty_like(a)
        kv.prefill_batch_attn(c.q, c.k_new, c.v_new, i32(range(100, 100 + n)),
                              c.slots.repeat(n), c.qw, c.kw, c.inv_freq, None, out, c.eps, c.scale)
        assert torch.equal(K, c.K) and torch.equal(V, c.V)
        assert float((out - a).abs().max()) <= 1e-5
        kv.free()


def test_empty_requests_and_empty_calls():
    par = [-1, 0]
    c = Case([(10, []), (50, par), (7, []), (300, [-1]), (2, [])], 1, 2, 64, pad=4)
    go(c)
    kv = SlotKV(4, 100, 1, 64, 4, 2)
    z = torch.empty(0, 2, 64, device="cuda")
    k = torch.empty(0, 1, 64, device="cuda")
    w, f = torch.ones(64, device="cuda"), torch.ones(32, device="cuda")
    for R in (0, 2):
        kv.tree_batch_attn(z, k, k, i32([0] * R), i32([1] * R), i32([0] * (R + 1)), i32([]), w, w, f,
                           None, None, z, 1e-6, 0.1)
    assert kv.get_status() == 0
    kv.free()


def bad_case(block):
    par = [-1, 0, 0, 1, 2]
    return Case([(60, par), (130, par), (0, par), (90, par), (3, par)], 2, 2, 128, block=block,
                spare=0, pad=3)


@pytest.mark.parametrize("block", [0, 64])
@pytest.mark.parametrize("kind", ["where", "long", "parent_self", "parent_later", "parent_far", "shrinks",
                                  "past_rows"])
def test_requests_out_of_range(block, kind):
    """One request is refused, the others are as without it."""
    c = bad_case(block)
    K0, V0 = c.K.clone(), c.V.clone()
    r, skip = 3, {3}
    if kind == "where":
        if block:
            c.tables[r, 0] = c.K.shape[0]
        else:
            c.slots[r] = c.K.shape[0]
    elif kind == "long":
        c.past[r] = (c.tables.shape[1] * block if block else c.K.shape[1]) - 4
    elif kind.startswith("parent"):
        c.parents[15 + 2] = {"parent_self": 2, "parent_later": 3, "parent_far": -2}[kind]
    elif kind == "shrinks":
        c.starts[r + 1] = 14  # request 3 ends before it begins, 4 takes its rows too
        skip = {3, 4}
    else:
        c.starts[5] = 1 << 20
        skip, r = {4}, 4
    kv = c.handle()
    c.run(kv)
    if kind == "shrinks":
        torch.cuda.synchronize()
        assert kv.get_status() == skv.DEV_RANGE
        c.reqs = c.reqs[:3]
        c.rows = 15
        want = bad_case(block)
        want.run(kv2 := want.handle())
        assert float((c.out[:14] - want.out[:14]).abs().max()) <= 1e-5  # (split elsewhere)
        kv2.free()
    else:
        c.check(K0, V0, what=kind, skip=skip)
        assert kv.get_status() == skv.DEV_RANGE
    kv.free()


@pytest.mark.parametrize("past", [2**32 - 4, 2**32 - 2, 2**31 - 256, 2**31])
def test_places_past_32_bits_are_refused(past):
    """A table may name more places than 32 bits count; a request there is refused
    (its places' sum must not wrap), the other one is served."""
    c = Case([(5, [-1, 0, 1, 1]), (9, [-1, 0])], 1, 1, 64, block=64)
    K0, V0 = c.K.clone(), c.V.clone()
    wide = torch.zeros(2, 2**26 + 3, dtype=torch.int32, device="cuda")
    wide[:, :c.tables.shape[1]] = c.tables
    c.tables = wide
    c.past[0] = past if past < 2**31 else past - 2**32
    kv = c.handle()
    c.run(kv)
    c.check(K0, V0, skip={0})
    assert kv.get_status() == skv.DEV_RANGE
    want = c.K.clone()
    kv.keep_path_paged(c.tables, c.past, c.starts, i32([2, 1]), i32([0, 3, 0, 0, 0, 0]))
    assert kv.get_status() == skv.DEV_RANGE
    assert torch.equal(c.K, want)
    kv.free()


def test_more_nodes_than_a_tree_may_have():
    c = Case([(5, list(range(-1, 256))), (9, [-1, 0])], 1, 1, 64)
    K0, V0 = c.K.clone(), c.V.clone()
    kv = c.handle()
    c.run(kv)
    c.check(K0, V0, skip={0})
    assert kv.get_status() == skv.DEV_RANGE
    kv.free()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("block", [0, 64])
def test_many_requests(hd, block):
    """More requests than SMs, of every size, some without nodes."""
    r = random.Random(hd)
    lens = [(r.choice([0, 1, 40, 127, 128, 300]), r.choice([0, 1, 2, 5, 9])) for _ in range(400)]
    go(Case([(p, tree(r, n, 3)) for p, n in lens], 2, 2, hd, block=block, seed=1, pad=1))


def test_thousands_of_requests():
    """More than the planning looks at at once, many times over, of one block of rows and of several."""
    r = random.Random(2)
    lens = [(r.choice([0, 3, 130]), r.choice([0, 0, 1, 1, 2, 70 if i % 500 == 0 else 1])) for i in range(2500)]
    go(Case([(p, tree(r, n, 3)) for p, n in lens], 1, 2, 64, seed=4))


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_sums_do_not_shrink(hd):
    """The tensor core cuts every sum toward zero; what that takes on average is put back, so
    the outputs are not smaller than they should be by more than what the estimate leaves:
    of O 2 of up to 4 units of 2^-23, half a unit each of both roundings, of S a unit per
    e-fold of the scores here (log2 units up to 12 times 2^-24 ln 2): below 5e-7."""
    r = random.Random(hd)
    c = Case([(3000, tree(r, 20, 4)), (777, tree(r, 9, 2))], 2, 4, hd, seed=7)
    c.K *= 3.0
    K0, V0 = c.K.clone(), c.V.clone()
    kv = c.handle()
    c.run(kv)
    want = torch.stack(c.check(K0, V0)).flatten()
    got = c.out[:c.rows].double().flatten()
    assert abs(float(((got - want) * want).sum() / want.pow(2).sum())) <= 5e-7
    kv.free()


@pytest.mark.parametrize("hd,block", [(64, 0), (128, 128), (256, 0)])
def test_long_history(hd, block):
    """One request over many keys (split over the GPU), beside short ones."""
    r = random.Random(1)
    go(Case([(40, tree(r, 3, 2)), (20011, tree(r, 24, 6)), (77, tree(r, 5, 5))], 2, 4, hd, block=block,
            seed=3, sinks=True))


def test_captured_and_replayed():
    c = Case(requests(2, [(500, 16), (90, 7)]), 2, 4, 128, sinks=True)
    kv = c.handle()
    with pytest.raises(skv.SlotKVError, match="before"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(kv)
    del g
    c.run(kv)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.run(kv)
    for i in range(3):
        c.q.normal_()
        c.k_new.normal_()
        c.past.copy_(i32([500 - 7 * i, 90 + i]))
        c.reqs = [(500 - 7 * i, c.reqs[0][1]), (90 + i, c.reqs[1][1])]
        K0, V0 = c.K.clone(), c.V.clone()
        g.replay()
        c.check(K0, V0, what=f"replay {i}")
    kv.free()


def test_other_stream_and_repeats():
    c = Case(requests(5, [(700, 30), (2000, 50), (64, 1)]), 2, 4, 64)
    kv = c.handle()
    K0, V0 = c.K.clone(), c.V.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(kv, stream=s)
    s.synchronize()
    c.check(K0, V0)
    a = c.out.clone()
    for _ in range(20):  # the same bits every time
        c.run(kv)
    assert torch.equal(a, c.out)
    kv.free()


def test_two_handles_in_two_streams():
    """Two calls at once, each with its own handle."""
    cs = [Case(requests(i, [(900, 20), (33, 6)]), 2, 4, 128, seed=i) for i in range(2)]
    kvs = [c.handle() for c in cs]
    K0 = [(c.K.clone(), c.V.clone()) for c in cs]
    ss = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, kv, s in zip(cs, kvs, ss):
            c.run(kv, stream=s)
    torch.cuda.synchronize()
    for c, kv, (a, b) in zip(cs, kvs, K0):
        c.check(a, b)
        kv.free()


def test_both_ways_of_the_binding_agree(monkeypatch):
    """The compiled call and the ctypes one."""
    for block in (0, 64):
        c = Case(requests(5, [(200, 12), (31, 9)]), 2, 2, 128, block=block, slopes=True, docs=[3, 0])
        kv = c.handle()
        a = c.run(kv).clone()
        c.out.zero_()
        monkeypatch.setattr(skv, "_call", False)
        assert torch.equal(c.run(kv), a)
        monkeypatch.undo()
        kv.free()


def test_cache_past_32_bits():
    """A pool of more than 2^32 bytes, the request's blocks at its end."""
    hd, n_kv, block = 128, 8, 64
    n = (1 << 32) // (block * n_kv * hd * 4) + 40
    c = Case([(150, [-1, 0, 0])], n_kv, 2, hd, block=block)
    K, V = torch.zeros(n, block, n_kv, hd, device="cuda"), torch.zeros(n, block, n_kv, hd, device="cuda")
    m = c.K.shape[0]
    K[n - m:], V[n - m:] = c.K, c.V
    c.K, c.V, c.tables = K, V, c.tables + (n - m)
    kv = c.handle()
    K0, V0 = c.K.clone(), c.V.clone()
    c.run(kv)
    c.check(K0, V0)
    kv.free()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("past", [300, 30000])
def test_a_wait_that_runs_out_ends_the_call(hd, past):
    """The stalled pipeline (a signal withheld): the call ends by itself with the
    flag raised, and the handle works afterwards."""
    c = Case(requests(2, [(past, 16), (64, 7)]), 1, 4, hd)
    kv = c.handle()
    kv.set_options(skv.OPT_TEST_STALL)
    c.run(kv)
    assert kv.get_status() & skv.DEV_TIMEOUT
    kv.set_options(0)
    c.out.fill_(7.5)
    K0, V0 = c.K.clone(), c.V.clone()
    c.run(kv)
    c.check(K0, V0)
    assert kv.get_status() == 0
    kv.free()
