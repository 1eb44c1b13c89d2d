"""The scored calls (capped scores, distance bias, windows, document and
prefix masks) against their definition in 64 bits: decode over slots and a
paged pool, batched prefill, at the sizes and masks where they can go wrong."""
import math

import pytest
import torch

import sequence_slot_kv_gb300 as skv
from plain64 import F64, check, key_range, norm_rope, row_attention
from sequence_slot_kv_gb300 import Scores, SlotKV

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Layer:
    """A handle over random slots with a layer's parameters."""

    def __init__(self, n_slots, ctx, n_kv, G, hd, rows, seed=0, sinks=False, slopes=False):
        g = self.g = _gen(seed)
        self.n_kv, self.G, self.hd, self.n_head = n_kv, G, hd, n_kv * G
        self.K = torch.randn(n_slots, ctx, n_kv, hd, generator=g, device="cuda")
        self.V = torch.randn(n_slots, ctx, n_kv, hd, generator=g, device="cuda")
        self.kv = SlotKV(n_slots, ctx, n_kv, hd, rows, self.n_head, k_buf=self.K, v_buf=self.V)
        self.qw = 1 + 0.1 * self.rnd(hd)
        self.kw = 1 + 0.1 * self.rnd(hd)
        self.inv = (10000.0 ** (-2 * torch.arange(hd // 2, device="cuda", dtype=F64) / hd)).float()
        self.sinks = self.rnd(self.n_head) if sinks else None
        self.slopes = (2.0 ** (-6.0 * (torch.arange(self.n_head, device="cuda") + 1.0)
                               / self.n_head)).float() if slopes else None
        self.scale = hd ** -0.5

    def rnd(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def step(self, rows):
        return (self.rnd(rows, self.n_head, self.hd), self.rnd(rows, self.n_kv, self.hd),
                self.rnd(rows, self.n_kv, self.hd))

    def params(self):
        return self.qw, self.kw, self.inv, self.sinks


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def want_rows(L, q, k_new, v_new, pos, where, keys_of, prefill, cap=0.0, window=0, doc=None,
              pend=None, skip=()):
    """Expected K, V (f64 on the new rows), outputs and tolerances.  where[b]:
    (slot or block, place) of the new key; keys_of(b, lo, hi): index of keys
    lo .. hi of the row in K and V."""
    position = torch.tensor(pos, device="cuda")
    q64 = norm_rope(q, L.qw, position, L.inv, EPS)
    k64 = norm_rope(k_new, L.kw, position, L.inv, EPS)
    K, V = L.K.to(F64), L.V.to(F64)
    for b, (x, y) in enumerate(where):
        if b not in skip:
            K[x, y], V[x, y] = k64[b], v_new[b].to(F64)
    outs, tols = [], []
    for b, p in enumerate(pos):
        lo, hi = key_range(p, b, prefill, window, doc, pend)
        t = torch.arange(lo, max(lo, hi + 1), device="cuda")
        if b in skip or lo > hi:
            out, tol = torch.zeros(L.n_head, L.hd, dtype=F64, device="cuda"), 0.0
        else:
            sel = keys_of(b, t)
            out, tol = row_attention(q64[b], K[sel], V[sel], p, t,
                                     torch.ones(len(t), dtype=torch.bool, device="cuda"),
                                     L.scale, cap, L.slopes, L.sinks)
        outs.append(out)
        tols.append(tol)
    return K, V, outs, tols


def check_cache(L, K64, V64, where, skip=()):
    """New K rows within f32 rounding of the norm and rotation (8 ulp of the
    row's largest), new V rows and everything else to the bit."""
    K, V = L.K.to(F64), L.V.to(F64)
    for b, (x, y) in enumerate(where):
        if b in skip:
            continue
        err = (K[x, y] - K64[x, y]).abs().max()
        assert float(err) <= 2.0 ** -20 * float(K64[x, y].abs().max())
        K[x, y] = K64[x, y]
    same = (K == K64) | (torch.isnan(K) & torch.isnan(K64))
    assert bool(same.all()), "K changed outside the new rows"
    same = (V == V64) | (torch.isnan(V) & torch.isnan(V64))
    assert bool(same.all()), "V changed"


RULES = [dict(cap=30.0), dict(window=7), dict(slopes=True), dict(docs=True, sinks=True),
         dict(cap=5.0, window=100, slopes=True, docs=True, sinks=True)]


def decode_case(hd, G, n_kv, B, ctx, rule, seed, split=None, block=0, poison=True, pos=None):
    sinks, slopes = rule.get("sinks", False), rule.get("slopes", False)
    cap, window = rule.get("cap", 0.0), rule.get("window", 0)
    if block:
        per = -(-ctx // block)
        L = Layer(B * per + 1, block, n_kv, G, hd, B, seed, sinks, slopes)
        tab = torch.randperm(B * per + 1, generator=L.g, device="cuda")[:B * per].view(B, per)
    else:
        L = Layer(B + 1, ctx, n_kv, G, hd, B, seed, sinks, slopes)
        slots = torch.randperm(B + 1, generator=L.g, device="cuda")[:B]
    if split:
        L.kv.set_split(*split)
    r = torch.Generator().manual_seed(seed)
    if pos is None:
        pos = [0, ctx - 1] + torch.randint(0, ctx, (B,), generator=r).tolist()
        pos = pos[:B]
    doc = None
    if rule.get("docs"):
        doc = [int(torch.randint(0, p + 1, (1,), generator=r)) for p in pos]
        doc[-1] = pos[-1] + 3  # nothing left
        doc[0] = pos[0]        # only its own key
    q, k_new, v_new = L.step(B)
    if block:
        where = [(int(tab[b, p // block]), p % block) for b, p in enumerate(pos)]

        def keys_of(b, t):
            return tab[b, t // block], t % block
    else:
        where = [(int(slots[b]), p) for b, p in enumerate(pos)]

        def keys_of(b, t):
            return int(slots[b]), t
    if poison:  # NaN and infinities in every place the row does not attend
        for b, p in enumerate(pos):
            lo, _ = key_range(p, b, False, window, doc)
            for t in [*range(max(0, min(lo, p + 1) - 40), min(lo, p)), *range(p + 1, min(ctx, p + 40))]:
                x = keys_of(b, torch.tensor(t, device="cuda"))
                L.K[x], L.V[x] = (math.nan, math.inf) if t % 2 else (math.inf, math.nan)
    K64, V64, outs, tols = want_rows(L, q, k_new, v_new, pos, where, keys_of, False, cap, window,
                                     doc)
    out = torch.full((B, L.n_head, hd), math.nan, device="cuda")
    sc = Scores(cap, window, L.slopes, i32(doc) if doc else None)
    if block:
        tables = tab.to(torch.int32).clone()
        for b, p in enumerate(pos):  # entries outside the row's used blocks are never read
            lo, _ = key_range(p, b, False, window, doc)
            tables[b, p // block + 1:] = -1
            tables[b, :min(lo, p) // block] = -1
        L.kv.decode_batch_attn_paged_scored(q, k_new, v_new, i32(pos), tables, *L.params(), sc,
                                            out, EPS, L.scale)
    else:
        L.kv.decode_batch_attn_scored(q, k_new, v_new, i32(pos), slots.to(torch.int32),
                                      *L.params(), sc, out, EPS, L.scale)
    assert L.kv.get_status() == 0
    check(out, outs, tols, "decode")
    check_cache(L, K64, V64, where)
    L.kv.free()


@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("hd,G", [(64, 1), (64, 8), (128, 2), (128, 3), (256, 1), (256, 5)])
def test_decode_small_calls(hd, G, rule):
    decode_case(hd, G, 2, 5, 230, rule, seed=hd + G)


@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("hd,G,split", [(64, 4, (64, 8)), (128, 1, (32, 16)), (128, 8, (64, 4)),
                                        (256, 2, (16, 64)), (256, 8, (32, 3))])
def test_decode_split_rows(hd, G, split, rule):
    decode_case(hd, G, 2, 6, 900, rule, seed=3 * hd + G, split=split)


@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_decode_every_head_layout(hd, G):
    decode_case(hd, G, 3, 4, 700, RULES[4], seed=7 * hd + G)


@pytest.mark.parametrize("rule", RULES, ids=str)
@pytest.mark.parametrize("hd,G,ctx,block,split", [(64, 4, 256, 64, None), (128, 2, 1500, 64, (32, 8)),
                                                  (128, 5, 200, 32, None), (256, 1, 900, 16, (16, 16)),
                                                  (256, 4, 600, 48, None)])
def test_decode_paged(hd, G, ctx, block, split, rule):
    decode_case(hd, G, 2, 6, ctx, rule, seed=5 * hd + G, split=split, block=block)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 65, 1 << 31, (1 << 32) - 1])
def test_decode_window_borders(window):
    decode_case(128, 2, 1, 4, 400, dict(window=window), seed=window & 255, split=(32, 4),
                pos=[0, window % 400, 63, 399])


def test_decode_many_rows():
    """More (row, kv head) pairs than CTAs: items from the plan's list."""
    decode_case(64, 2, 4, 200, 300, RULES[4], seed=9, split=(64, 4), poison=False)


def test_decode_large_slopes_and_caps():
    """Slopes whose bias passes f32's range, and caps far above and below the scores."""
    for cap in (1e-3, 1e6):
        L = Layer(3, 500, 1, 4, 64, 2, seed=2)
        L.slopes = torch.tensor([0.0, 1e30, 1e38, 3.0], device="cuda")
        pos, q = [499, 320], L.step(2)
        want = want_rows(L, *q, pos, [(0, 499), (2, 320)], lambda b, t: ((0, 2)[b], t), False, cap)
        out = torch.full((2, 4, 64), math.nan, device="cuda")
        L.kv.decode_batch_attn_scored(*q, i32(pos), i32([0, 2]), *L.params(),
                                      Scores(cap, 0, L.slopes), out, EPS, L.scale)
        check(out, want[2], want[3], "decode")
        L.kv.free()


def test_no_rule_is_the_plain_call():
    """Scores() and None give the plain calls' results, to the bit in a decode."""
    L = Layer(6, 1000, 2, 4, 128, 40, seed=4, sinks=True)
    q, pos, slots = L.step(5), i32([0, 5, 999, 400, 64]), i32([5, 1, 0, 3, 2])
    outs = []
    for sc in (None, Scores(), "plain"):
        out = torch.full((5, 8, 128), math.nan, device="cuda")
        if sc == "plain":
            L.kv.decode_batch_attn(*q, pos, slots, *L.params(), out, EPS, L.scale)
        else:
            L.kv.decode_batch_attn_scored(*q, pos, slots, *L.params(), sc, out, EPS, L.scale)
        outs.append(out)
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])
    L.kv.free()


@pytest.mark.parametrize("hd,block", [(64, 0), (256, 0), (128, 64)])
def test_decode_rows_out_of_range(hd, block):
    """Bad slots, positions and table entries: flagged, skipped, nothing written."""
    L = Layer(8, block or 96, 2, 2, hd, 4, seed=6)
    K0, V0 = L.K.clone(), L.V.clone()
    q, out = L.step(4), torch.full((4, 4, hd), 7.0, device="cuda")
    sc = Scores(cap=20.0, doc_start=i32([0, 0, 9, 0]))
    if block:
        tables = i32([[0, 1], [2, 9], [3, 4], [5, -1]])  # row 1's second block is no block
        pos = [100, 100, 128, 70]                        # row 2 is past its table, row 3 uses -1
        L.kv.decode_batch_attn_paged_scored(*q, i32(pos), tables, *L.params(), sc, out, EPS,
                                            L.scale)
        good, place = [0], [(1, 100 - block)]
    else:
        pos = [5, 96, 10, 95]
        L.kv.decode_batch_attn_scored(*q, i32(pos), i32([0, 1, 8, 2]), *L.params(), sc, out, EPS,
                                      L.scale)
        good, place = [0, 3], [(0, 5), (2, 95)]
    assert L.kv.get_status() == skv.DEV_RANGE
    for b in range(4):
        assert bool((out[b] == 7.0).all()) == (b not in good)
    for x, y in place:
        K0[x, y], V0[x, y] = L.K[x, y], L.V[x, y]
    assert torch.equal(K0, L.K) and torch.equal(V0, L.V)
    L.kv.free()


# ------------------------------------------------------------------ prefill
def prefill_case(hd, G, n_kv, seqs, ctx, rule, seed, poison=True, order=None, pad=0):
    """seqs: (past, fresh) per sequence; order: a permutation seed of the tokens;
    pad: rows of no slot after the others."""
    sinks, slopes = rule.get("sinks", False), rule.get("slopes", False)
    cap, window = rule.get("cap", 0.0), rule.get("window", 0)
    n = sum(f for _, f in seqs)
    L = Layer(len(seqs) + 1, ctx, n_kv, G, hd, n + pad + 3, seed, sinks, slopes)
    r = torch.Generator().manual_seed(seed)
    toks = [(s + 1, p) for s, (past, f) in enumerate(seqs) for p in range(past, past + f)]
    if order is not None:
        toks = [toks[i] for i in torch.randperm(n, generator=torch.Generator().manual_seed(order))]
    pos = [p for _, p in toks]
    doc = pend = None
    ends = {s + 1: past + f for s, (past, f) in enumerate(seqs)}
    if rule.get("docs"):
        cuts = {s: sorted({0, *torch.randint(0, e, (3,), generator=r).tolist()})
                for s, e in ends.items()}
        doc = [max(c for c in cuts[s] if c <= p) for s, p in toks]
        doc[0] = pos[0] + 1 if not rule.get("prefix") else doc[0]  # nothing left
    if rule.get("prefix"):
        pe = {s: int(torch.randint(1, e + 1, (1,), generator=r)) for s, e in ends.items()}
        pend = [pe[s] if p < pe[s] else 0 for s, p in toks]
    q, k_new, v_new = L.step(n)
    where = [(s, p) for s, p in toks]
    if poison:  # whatever lies past the sequences, or before every row's keys
        for s, e in ends.items():
            lows = [key_range(p, b, True, window, doc, pend)[0] for b, (x, p) in enumerate(toks) if x == s]
            past = seqs[s - 1][0]
            first = min(lows)
            L.K[s, e:], L.V[s, e:] = math.nan, math.inf
            L.K[s, :min(first, past)], L.V[s, :min(first, past)] = math.inf, math.nan
    K64, V64, outs, tols = want_rows(L, q, k_new, v_new, pos, where, lambda b, t: (toks[b][0], t),
                                     True, cap, window, doc, pend)
    more = lambda x: torch.cat([x, x[:1].expand(pad, *x.shape[1:])]).contiguous() if pad else x
    rows = lambda x: i32(x + [0] * pad) if x else None
    out = torch.full((n + pad, L.n_head, hd), math.nan, device="cuda")
    sc = Scores(cap, window, L.slopes, rows(doc), rows(pend))
    L.kv.prefill_batch_attn_scored(more(q), more(k_new), more(v_new), rows(pos),
                                   i32([s for s, _ in toks] + [-1] * pad), *L.params(), sc, out,
                                   EPS, L.scale)
    assert L.kv.get_status() == (1 if pad else 0)
    check(out, outs, tols, "prefill")
    assert bool(torch.isnan(out[n:]).all()), "a row of no slot was written"
    check_cache(L, K64, V64, where)
    L.kv.free()


PREFILL_RULES = RULES + [dict(prefix=True), dict(prefix=True, cap=8.0, slopes=True, window=90,
                                                 docs=True, sinks=True)]


@pytest.mark.parametrize("rule", PREFILL_RULES, ids=str)
@pytest.mark.parametrize("hd,G", [(64, 1), (64, 4), (64, 7), (128, 2), (128, 8), (128, 3), (256, 2)])
def test_prefill(hd, G, rule):
    prefill_case(hd, G, 2, [(0, 70), (130, 33), (5, 1)], 200, rule, seed=hd + G)


@pytest.mark.parametrize("G", range(1, 9))
@pytest.mark.parametrize("hd", [64, 128])
def test_prefill_every_head_layout(hd, G):
    prefill_case(hd, G, 1, [(40, 130)], 190, PREFILL_RULES[-1], seed=hd * 3 + G)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rule", [PREFILL_RULES[-1], dict(cap=10.0), dict(window=300)], ids=str)
def test_prefill_split_over_a_long_history(hd, rule):
    """One token, one tile, an odd tile count: a long history cut into splits."""
    for fresh in (1, 31, 77):
        prefill_case(hd, 4, 1, [(2100, fresh)], 2200, rule, seed=hd + fresh)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prefill_tokens_in_any_order(hd):
    prefill_case(hd, 2, 2, [(0, 40), (20, 50), (300, 9)], 400, PREFILL_RULES[-1], seed=hd, order=3)


@pytest.mark.parametrize("hd,G", [(64, 8), (128, 8), (64, 1)])
def test_prefill_of_a_padded_batch(hd, G):
    """A call padded with rows of no slot, as one of fixed capacity is: enough
    rows that it would not be split, too few tokens not to be."""
    prefill_case(hd, G, 8 if G == 8 else 2, [(900, 21), (0, 3)], 1000, dict(cap=12.0, window=600),
                 seed=hd + G, pad=5000 if G == 1 else 900)


def test_prefill_of_many_tokens():
    """More tokens than one round of the plan takes, most sequences short."""
    prefill_case(64, 1, 1, [(3, 5)] * 1500 + [(0, 790), (40, 150)], 800, dict(window=50, slopes=True),
                 seed=5, poison=False)


@pytest.mark.parametrize("hd", [64, 128])
def test_prefill_not_split(hd):
    """Enough tiles that nothing is split."""
    prefill_case(hd, 1, 8, [(0, 150)] * 20, 150, dict(cap=20.0, docs=True), seed=hd, poison=False)


@pytest.mark.parametrize("hd,past", [(64, 0), (128, 0), (128, 1500), (64, 1500), (256, 0)])
def test_prefill_infinities_of_another_document(hd, past):
    """V of one document holds infinities and NaN, in the same tiles as the
    next document's rows: they reach the first one's rows only."""
    n, cut = 60, past + 25
    L = Layer(2, past + 100, 1, 2, hd, n, seed=8)
    pos = list(range(past, past + n))
    doc = [0 if p < cut else cut for p in pos]
    q, k_new, v_new = L.step(n)
    v_new[5, 0, 3] = math.inf
    v_new[6, 0, 9] = math.nan
    v_new[7, 0, 11] = -math.inf
    where = [(1, p) for p in pos]
    K64, V64, outs, tols = want_rows(L, q, k_new, v_new, pos, where, lambda b, t: (1, t), True,
                                     doc=doc)
    out = torch.full((n, 2, hd), math.nan, device="cuda")
    L.kv.prefill_batch_attn_scored(q, k_new, v_new, i32(pos), i32([1] * n), *L.params(),
                                   Scores(doc_start=i32(doc)), out, EPS, L.scale)
    assert not bool(torch.isfinite(outs[10]).all()) and bool(torch.isfinite(outs[30]).all())
    check(out, outs, tols, "prefill")
    L.kv.free()


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prefill_rows_out_of_range(hd):
    """A bad slot, position or prefix end: that token is skipped, the others see
    neither it nor its key; a prefix past the slot writes nothing."""
    L = Layer(3, 64, 2, 2, hd, 8, seed=11)
    pos, slots = [3, 64, 4, 5, 6, 0], [1, 1, 9, 1, 1, 2]
    pend = [0, 0, 0, 65, 0, 64]
    skip = (1, 2, 3)
    K0, V0 = L.K.clone(), L.V.clone()
    q, k_new, v_new = L.step(6)
    where = [(s if b not in skip else 0, p if b not in skip else 0)
             for b, (s, p) in enumerate(zip(slots, pos))]
    K64, V64, outs, tols = want_rows(L, q, k_new, v_new, pos, where, lambda b, t: (slots[b], t),
                                     True, pend=pend, skip=skip)
    out = torch.full((6, 4, hd), 7.0, device="cuda")
    L.kv.prefill_batch_attn_scored(q, k_new, v_new, i32(pos), i32(slots), *L.params(),
                                   Scores(prefix_end=i32(pend)), out, EPS, L.scale)
    assert L.kv.get_status() == skv.DEV_RANGE
    for b in skip:
        assert bool((out[b] == 7.0).all())
        outs[b] = out[b].to(F64)
    check(out, outs, tols, "prefill")
    check_cache(L, K64, V64, where, skip)
    L.kv.free()


def test_prefill_empty_call():
    L = Layer(2, 64, 1, 1, 64, 4, seed=1)
    e = torch.empty(0, 1, 64, device="cuda")
    L.kv.prefill_batch_attn_scored(e, e, e, i32([]), i32([]), *L.params(), Scores(cap=3.0), e, EPS,
                                   L.scale)
    L.kv.decode_batch_attn_scored(e, e, e, i32([]), i32([]), *L.params(), Scores(cap=3.0), e, EPS,
                                  L.scale)
    assert L.kv.get_status() == 0
    L.kv.free()


# ------------------------------------------------------------------ graphs, streams
@pytest.mark.parametrize("hd", [64, 128])
def test_captured_calls_replay(hd):
    """A prefill and a decode step captured together (after one call of each
    kind), replayed on another stream's work, equal to the eager ones."""
    L = Layer(4, 800, 2, 4, hd, 60, seed=hd, sinks=True, slopes=True)
    n = 60
    pos = i32(list(range(700, 700 + n)))
    slots = i32([2] * n)
    q, dq = L.step(n), L.step(3)
    dpos, dslots = i32([799, 10, 300]), i32([0, 1, 3])
    sc = Scores(cap=9.0, window=333, slopes=L.slopes)
    outs = [torch.zeros(n, 8, hd, device="cuda"), torch.zeros(3, 8, hd, device="cuda")]

    def both():
        L.kv.prefill_batch_attn_scored(*q, pos, slots, *L.params(), sc, outs[0], EPS, L.scale)
        L.kv.decode_batch_attn_scored(*dq, dpos, dslots, *L.params(), sc, outs[1], EPS, L.scale)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with pytest.raises(skv.SlotKVError, match="before"):  # nothing allocated yet
        with torch.cuda.stream(s):
            g.capture_begin(capture_error_mode="relaxed")
            try:
                both()
            finally:
                g.capture_end()
    both()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both()
    for o in outs:
        o.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    with torch.cuda.stream(s):
        for o in outs:
            o.zero_()
        both()
    s.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    L.kv.free()


@pytest.mark.parametrize("compiled", [True, False])
def test_both_ways_a_call_is_made(compiled, monkeypatch):
    """The compiled calls and the ctypes ones take the same arguments and give
    the same results; wrong arguments get the same errors from both."""
    assert skv._compiled(), "the compiled calls are not built"
    if not compiled:
        monkeypatch.setattr(skv, "_call", False)
    L = Layer(4, 128, 2, 2, 64, 6, seed=31, sinks=True, slopes=True)
    pos, slots, doc = [5, 90, 127], [3, 0, 1], [0, 80, 3]
    q = L.step(3)
    sc = Scores(7.0, 60, L.slopes, i32(doc))
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        K64, V64, outs, tols = want_rows(L, *q, pos, list(zip(slots, pos)),
                                         lambda b, t: (slots[b], t), False, 7.0, 60, doc)
        out = torch.full((3, 4, 64), math.nan, device="cuda")
        torch.cuda.synchronize()
        L.kv.decode_batch_attn_scored(*q, i32(pos), i32(slots), *L.params(), sc, out, EPS,
                                      L.scale, stream)
        torch.cuda.synchronize()
        check(out, outs, tols, "decode")
    bad = [(ValueError, dict(out=out[:2])), (TypeError, dict(out=out.double())),
           (ValueError, dict(out=out.transpose(1, 2))), (ValueError, dict(out=out.cpu())),
           (ValueError, dict(scores=Scores(doc_start=i32(doc + [0])))),
           (ValueError, dict(scores=Scores(slopes=L.slopes[:2]))),
           (skv.SlotKVError, dict(scores=Scores(cap=-1.0))),
           (skv.SlotKVError, dict(scores=Scores(cap=math.nan))),
           (skv.SlotKVError, dict(scores=Scores(cap=1e9))),
           (skv.SlotKVError, dict(scores=Scores(prefix_end=i32(doc)))),
           (ValueError, dict(q=None))]
    good = dict(q=q[0], k_new=q[1], v_new=q[2], positions=i32(pos), slots=i32(slots),
                q_norm_w=L.qw, k_norm_w=L.kw, inv_freq=L.inv, sinks=L.sinks, scores=sc, out=out,
                eps=EPS, scale=L.scale)
    for err, change in bad:
        with pytest.raises(err):
            L.kv.decode_batch_attn_scored(**{**good, **change})
    with pytest.raises(ValueError, match="block_tables"):
        L.kv.decode_batch_attn_paged_scored(
            **{k: v for k, v in good.items() if k != "slots"}, block_tables=i32(slots))
    with pytest.raises(skv.SlotKVError, match="kv heads"):
        other = SlotKV(1, 128, 1, 64, 1, 2)
        L.kv.decode_batch_attn_shared(**good, prefix=other, prefix_slots=i32([0] * 3),
                                      prefix_lens=i32([0] * 3))
    wide = Layer(1, 64, 1, 1, 256, 1)
    one = wide.step(1)
    with pytest.raises(skv.SlotKVError, match="head_dim"):
        wide.kv.decode_batch_attn_shared(*one, i32([0]), i32([0]), wide.kv, i32([0]), i32([0]),
                                         *wide.params(), None, torch.empty(1, 1, 256, device="cuda"),
                                         EPS, 1.0)
    for h in (L.kv, wide.kv):
        h.free()
    with pytest.raises(skv.SlotKVError, match="not allocated"):
        L.kv.decode_batch_attn_scored(**good)
