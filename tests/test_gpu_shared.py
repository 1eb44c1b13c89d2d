"""The shared-prefix decode step against its definition in 64 bits, and a run
of the request-length calls, the scored prefill and the shared step together."""
import math

import pytest
import torch

import sequence_slot_kv_gb300 as skv
from plain64 import F64, check, key_range, norm_rope, row_attention
from sequence_slot_kv_gb300 import Scores, SlotKV
from test_gpu_scored import EPS, Layer, check_cache, i32

pytestmark = pytest.mark.gpu


def shared_want(L, PK, PV, q, k_new, v_new, pos, slots, psl, plen, cap=0.0, window=0, doc=None,
                skip=()):
    position = torch.tensor(pos, device="cuda")
    q64 = norm_rope(q, L.qw, position, L.inv, EPS)
    k64 = norm_rope(k_new, L.kw, position, L.inv, EPS)
    K, V = L.K.to(F64), L.V.to(F64)
    where = [(s, p - n) for s, p, n in zip(slots, pos, plen)]
    for b, (x, y) in enumerate(where):
        if b not in skip:
            K[x, y], V[x, y] = k64[b], v_new[b].to(F64)
    outs, tols = [], []
    for b, p in enumerate(pos):
        if b in skip:
            outs.append(torch.zeros(L.n_head, L.hd, dtype=F64, device="cuda"))
            tols.append(0.0)
            continue
        n, (x, y) = plen[b], where[b]
        keys = [K[x, :y + 1]] if not n else [PK[psl[b], :n].to(F64), K[x, :y + 1]]
        vals = [V[x, :y + 1]] if not n else [PV[psl[b], :n].to(F64), V[x, :y + 1]]
        t = torch.arange(p + 1, device="cuda")
        lo, _ = key_range(p, b, False, window, doc)
        out, tol = row_attention(q64[b], torch.cat(keys), torch.cat(vals), p, t, t >= lo, L.scale,
                                 cap, L.slopes, L.sinks)
        outs.append(out)
        tols.append(tol)
    return K, V, outs, tols, where


def shared_case(hd, G, n_kv, groups, ctx, pctx, rule, seed, shuffle=False, split=None, rows=None):
    """groups: (prefix length, rows) each; length 0: plain rows."""
    sinks, slopes = rule.get("sinks", False), rule.get("slopes", False)
    cap, window = rule.get("cap", 0.0), rule.get("window", 0)
    B = sum(r for _, r in groups)
    L = Layer(B + 2, ctx, n_kv, G, hd, rows or B, seed, sinks, slopes)
    n_pre = len(groups) + 1
    PK, PV = L.rnd(n_pre, pctx, n_kv, hd), L.rnd(n_pre, pctx, n_kv, hd)
    pkv = SlotKV(n_pre, pctx, n_kv, hd, 1, L.n_head, k_buf=PK, v_buf=PV)
    if split:
        L.kv.set_split(*split)
    r = torch.Generator().manual_seed(seed)
    psl, plen = [], []
    for g, (n, c) in enumerate(groups):
        for j in range(c):
            psl.append(g + 1 if n else n_pre + 50)  # (not read without a prefix)
            # rows of one slot may use different lengths of it
            plen.append(n if j % 3 or not rule.get("ragged") else max(0, n - 5 * j))
    own = torch.randint(0, ctx, (B,), generator=r).tolist()
    own[0], own[-1] = 0, ctx - 1
    perm = torch.randperm(B, generator=r).tolist() if shuffle else list(range(B))
    psl, plen = [psl[i] for i in perm], [plen[i] for i in perm]
    pos = [a + b for a, b in zip(plen, own)]
    slots = (torch.randperm(B + 2, generator=r)[:B]).tolist()
    doc = None
    if rule.get("docs"):
        doc = [int(torch.randint(0, p + 1, (1,), generator=r)) for p in pos]
        doc[0] = pos[0] + 1
    q, k_new, v_new = L.step(B)
    # nothing past a prefix's or a row's keys may matter
    for g, (n, _) in enumerate(groups):
        PK[g + 1, n:], PV[g + 1, n:] = math.nan, math.inf
    for s, o in zip(slots, own):
        L.K[s, o:], L.V[s, o:] = math.inf, math.nan
    K64, V64, outs, tols, where = shared_want(L, PK, PV, q, k_new, v_new, pos, slots, psl, plen,
                                              cap, window, doc)
    P0 = PK.clone(), PV.clone()
    out = torch.full((B, L.n_head, hd), math.nan, device="cuda")
    sc = Scores(cap, window, L.slopes, i32(doc) if doc else None)
    for _ in range(2):  # a second call on the same workspace
        L.kv.decode_batch_attn_shared(q, k_new, v_new, i32(pos), i32(slots), pkv, i32(psl),
                                      i32(plen), *L.params(), sc if rule else None, out, EPS,
                                      L.scale)
        assert L.kv.get_status() == 0 and pkv.get_status() == 0
        check(out, outs, tols, "shared")
    check_cache(L, K64, V64, where)
    same = [(a == b) | (torch.isnan(a) & torch.isnan(b)) for a, b in zip(P0, (PK, PV))]
    assert all(bool(x.all()) for x in same)
    L.kv.free()
    pkv.free()


RULES = [{}, dict(sinks=True, ragged=True), dict(cap=6.0, slopes=True),
         dict(window=150, sinks=True), dict(cap=20.0, slopes=True, docs=True, sinks=True, ragged=True)]


@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("hd,G", [(64, 1), (64, 4), (64, 8), (128, 2), (128, 4), (128, 5)])
def test_shared(hd, G, rule):
    shared_case(hd, G, 2, [(300, 7), (0, 3), (64, 2), (1, 1), (200, 5)], 90, 310, rule,
                seed=hd + G)


@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("hd", [64, 128])
def test_shared_every_head_layout(hd, G):
    shared_case(hd, G, 1, [(700, 40)], 40, 700, RULES[4], seed=hd * 5 + G)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rule", [RULES[0], RULES[4]], ids=str)
def test_shared_long_prefix_split(hd, rule):
    """One kv head and few rows: the prefix is cut into many splits; own keys
    long enough for the persistent decode kernel, cut as well."""
    shared_case(hd, 4, 1, [(5000, 9)], 700, 5000, rule, seed=hd, split=(64, 4))


@pytest.mark.parametrize("hd", [64, 128])
def test_shared_rows_in_any_order(hd):
    shared_case(hd, 2, 2, [(130, 9), (0, 4), (260, 8)], 60, 260, RULES[4], seed=hd, shuffle=True)


def test_shared_many_rows():
    """More tiles than are ever split."""
    shared_case(64, 8, 8, [(96, 150), (64, 150), (80, 330)], 20, 96, RULES[2], seed=3)


def test_shared_prefix_in_the_same_handle():
    """The prefix handle may be the rows' own; a row may go on in its prefix's slot."""
    L = Layer(5, 400, 2, 4, 64, 3, seed=5)
    pos, slots, psl, plen = [200, 230, 210], [1, 2, 3], [0, 0, 0], [200, 200, 150]
    q = L.step(3)
    K0, V0 = L.K.clone(), L.V.clone()
    K64, V64, outs, tols, where = shared_want(L, K0, V0, *q, pos, slots, psl, plen)
    out = torch.full((3, 8, 64), math.nan, device="cuda")
    L.kv.decode_batch_attn_shared(*q, i32(pos), i32(slots), L.kv, i32(psl), i32(plen), *L.params(),
                                  None, out, EPS, L.scale)
    assert L.kv.get_status() == 0
    check(out, outs, tols, "shared")
    check_cache(L, K64, V64, where)
    L.kv.free()


def test_shared_infinities_in_the_prefix():
    """An infinite V of the prefix reaches the rows that attend its key only."""
    L = Layer(6, 64, 1, 4, 64, 5, seed=6)
    PK, PV = L.rnd(1, 300, 1, 64), L.rnd(1, 300, 1, 64)
    PV[0, 170, 0, 5], PV[0, 40, 0, 6] = math.inf, math.nan
    pkv = SlotKV(1, 300, 1, 64, 1, 4, k_buf=PK, v_buf=PV)
    plen = [300, 170, 171, 40, 300]
    pos = [n + 10 for n in plen]
    doc = [0, 0, 0, 0, 180]
    q = L.step(5)
    K64, V64, outs, tols, where = shared_want(L, PK, PV, *q, pos, [0, 1, 2, 3, 4], [0] * 5, plen,
                                              doc=doc)
    out = torch.full((5, 4, 64), math.nan, device="cuda")
    L.kv.decode_batch_attn_shared(*q, i32(pos), i32([0, 1, 2, 3, 4]), pkv, i32([0] * 5), i32(plen),
                                  *L.params(), Scores(doc_start=i32(doc)), out, EPS, L.scale)
    assert bool(torch.isinf(outs[2]).any()) and bool(torch.isfinite(outs[4]).all())
    check(out, outs, tols, "shared")
    L.kv.free()
    pkv.free()


def test_shared_rows_out_of_range():
    L = Layer(6, 32, 2, 2, 128, 8, seed=7)
    PK, PV = L.rnd(2, 100, 2, 128), L.rnd(2, 100, 2, 128)
    pkv = SlotKV(2, 100, 2, 128, 1, 4, k_buf=PK, v_buf=PV)
    #       fine  slot  pos<len own ctx  len>ctx  prefix slot  fine, none
    slots = [0, 6, 1, 2, 3, 4, 5]
    plen = [100, 50, 50, 50, 101, 50, 0]
    psl = [1, 0, 0, 0, 0, 2, 77]
    pos = [131, 60, 49, 82, 110, 60, 31]
    skip = (1, 2, 3, 4, 5)
    q = L.step(7)
    w_slots = [s if b not in skip else 0 for b, s in enumerate(slots)]
    K64, V64, outs, tols, where = shared_want(L, PK, PV, *q, pos, w_slots, psl, plen, skip=skip)
    out = torch.full((7, 4, 128), 7.0, device="cuda")
    L.kv.decode_batch_attn_shared(*q, i32(pos), i32(slots), pkv, i32(psl), i32(plen), *L.params(),
                                  None, out, EPS, L.scale)
    assert L.kv.get_status() == skv.DEV_RANGE and pkv.get_status() == 0
    for b in skip:
        assert bool((out[b] == 7.0).all())
        outs[b] = out[b].to(F64)
    check(out, outs, tols, "shared")
    check_cache(L, K64, V64, where, skip)
    L.kv.free()
    pkv.free()


def test_shared_captured_steps_replay():
    """Steps captured into two graphs of different batches on one handle,
    replayed in turn, with positions advanced on the device."""
    L = Layer(8, 64, 2, 4, 128, 6, seed=12)
    PK, PV = L.rnd(1, 500, 2, 128), L.rnd(1, 500, 2, 128)
    pkv = SlotKV(1, 500, 2, 128, 1, 8, k_buf=PK, v_buf=PV)
    batches = []
    for n, first in ((6, 0), (2, 6)):
        batches.append(dict(q=L.step(n), pos=i32([480 + j for j in range(n)]), first=first, n=n,
                            slots=i32(list(range(first, first + n))), psl=i32([0] * n),
                            plen=i32([480] * n), out=torch.zeros(n, 8, 128, device="cuda")))

    def step(x):
        L.kv.decode_batch_attn_shared(*x["q"], x["pos"], x["slots"], pkv, x["psl"], x["plen"],
                                      *L.params(), None, x["out"], EPS, L.scale)
        skv.slot_kv_advance_positions(x["pos"], 1)

    K0, V0 = L.K.clone(), L.V.clone()
    want = []
    for x in batches:
        p0 = x["pos"].clone()
        for _ in range(3):
            step(x)
        want.append(x["out"].clone())
        x["pos"].copy_(p0)
    torch.cuda.synchronize()
    K1, V1 = L.K.clone(), L.V.clone()
    L.K.copy_(K0)
    L.V.copy_(V0)
    graphs = []
    for x in batches:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(x)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert L.kv.get_status() == 0
    for x, w in zip(batches, want):
        assert torch.equal(x["out"], w)
    assert torch.equal(L.K, K1) and torch.equal(L.V, V1)
    L.kv.free()
    pkv.free()


def test_requests_from_prompt_to_shared_steps():
    """As a server uses them: a system prompt prefilled once, requests' token
    maps built on the device, their own prompts prefilled behind nothing (own
    slots), then decode steps on the shared prefix; and the same requests in a
    paged pool whose tables the device extends, which must agree."""
    hd, n_kv, G, bs, sys_len, R = 64, 2, 4, 64, 150, 3
    n_head, cap = n_kv * G, 15.0
    L = Layer(R, 256, n_kv, G, hd, 200, seed=21)          # the rows' own slots
    pre = SlotKV(1, 256, n_kv, hd, 200, n_head)            # the system prompt
    sc = Scores(cap=cap)
    q, k, v = L.step(sys_len)
    dev = dict(dtype=torch.int32, device="cuda")
    starts, ts, tp = torch.empty(2, **dev), torch.empty(sys_len, **dev), torch.empty(sys_len, **dev)
    pre.token_map(i32([0]), i32([0]), i32([sys_len]), starts, ts, tp)
    out = torch.empty(sys_len, n_head, hd, device="cuda")
    pre.prefill_batch_attn_scored(q, k, v, tp, ts, *L.params(), sc, out, EPS, L.scale)
    PK, PV = pre.kv_tensors()
    # the paged pool holds a copy of the prompt per request
    per = 4
    pool = Layer(R * per, bs, n_kv, G, hd, R, seed=22)
    tables = torch.full((R, per), -1, **dev)
    free, head = torch.randperm(R * per, device="cuda").to(torch.int32), i32([0])
    past = i32([0] * R)
    pool.kv.extend_tables(past, i32([sys_len] * R), tables, free, head)
    for r in range(R):
        for t0 in range(0, sys_len, bs):
            n = min(bs, sys_len - t0)
            b = int(tables[r, t0 // bs])
            pool.K[b, :n], pool.V[b, :n] = PK[0, t0:t0 + n], PV[0, t0:t0 + n]
    past.fill_(sys_len)
    pos, one = past.clone(), i32([1] * R)
    o1 = torch.empty(R, n_head, hd, device="cuda")
    o2 = torch.empty_like(o1)
    for step in range(50):
        q, k, v = L.step(R)
        L.kv.decode_batch_attn_shared(q, k, v, pos, i32([2, 0, 1]), pre, i32([0] * R),
                                      i32([sys_len] * R), *L.params(), sc, o1, EPS, L.scale)
        pool.kv.extend_tables(pos, one, tables, free, head)
        pool.kv.decode_batch_attn_paged_scored(q, k, v, pos, tables, *L.params(), sc, o2, EPS,
                                               L.scale)
        # both within the bound of the definition, so within twice of one
        # another: scores up to sqrt(hd) * 1.4^2 in |q||k|, |V| up to 5
        S = math.sqrt(hd) * 2.0
        tol = 2 * 5.0 * (2 * S * 3 * 2.0 ** -21 + 2 * cap * 2.0 ** -22 + 2.0 ** -19)
        assert float((o1 - o2).abs().max()) <= tol
        skv.slot_kv_advance_positions(pos, 1)
    assert L.kv.get_status() == 0 and pool.kv.get_status() == 0 and pre.get_status() == 0
    assert int(head) == R * math.ceil((sys_len + 50) / bs)
    for x in (L.kv, pool.kv, pre):
        x.free()


@pytest.mark.parametrize("hd", [64, 128])
def test_stalled_pipeline_times_out_and_recovers(hd):
    """The stall option withholds each CTA's first scores: a scored prefill and a
    shared step end with DEV_TIMEOUT after their bounded waits, and the handle
    works again."""
    L = Layer(4, 200, 1, 2, hd, 40, seed=17)
    PK, PV = L.rnd(1, 300, 1, hd), L.rnd(1, 300, 1, hd)
    pkv = SlotKV(1, 300, 1, hd, 1, 2, k_buf=PK, v_buf=PV)
    pos, slots, plen = [310, 305], [1, 2], [300, 300]
    q, pq = L.step(2), L.step(40)
    out, pout = torch.empty(2, 2, hd, device="cuda"), torch.empty(40, 2, hd, device="cuda")
    ppos, pslots = i32(list(range(40))), i32([3] * 40)

    def shared():
        L.kv.decode_batch_attn_shared(*q, i32(pos), i32(slots), pkv, i32([0, 0]), i32(plen),
                                      *L.params(), None, out, EPS, L.scale)

    def prefill():
        L.kv.prefill_batch_attn_scored(*pq, ppos, pslots, *L.params(), Scores(cap=9.0), pout, EPS,
                                       L.scale)

    for call in (shared, prefill):
        call()
        assert L.kv.get_status() == 0
        L.kv.set_options(skv.OPT_TEST_STALL)
        call()
        assert L.kv.get_status() & skv.DEV_TIMEOUT
        L.kv.set_options(0)
        call()
        assert L.kv.get_status() == 0
    K64, V64, outs, tols, where = shared_want(L, PK, PV, *q, pos, slots, [0, 0], plen)
    shared()
    check(out, outs, tols, "shared")
    L.kv.free()
    pkv.free()
