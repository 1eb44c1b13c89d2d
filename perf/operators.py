"""The operators of long shared serving contexts, as calls and in plain form.

Five operators that sit between a scheduler and the slot KV of this
framework, each with the cases it is measured on:

  * ``map``     request lengths -> one slot and position per prompt token
                (``slot_kv_token_map``, the input of a batched prefill);
  * ``tables``  request lengths -> block tables extended from a free list
                (``slot_kv_extend_tables``, the input of a paged decode step);
  * ``decode``  the decode step with capped scores, a distance bias, a window
                and document masks, over slots or over a paged pool
                (``decode_batch_attn_scored``, ``decode_batch_attn_paged_scored``);
  * ``prefill`` the batched prefill with the same, and prefix masks
                (``prefill_batch_attn_scored``);
  * ``shared``  the decode step of a batch whose rows share long prefixes, each
                prefix read once for all its rows (``decode_batch_attn_shared``).

With ``own`` false ``run`` is the plain form in elementary torch operations;
with ``own`` true it makes the framework's calls on the same state.
"""
import math
import random

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of chat requests joining a running batch: latency
        dict(name="map_few", kind="map", R=5, fresh=23, past=900, lens=1),
        # a prefill step of several hundred ragged prompts
        dict(name="map_prompts", kind="map", R=601, fresh=215, past=3000, lens=2),
        # one decode step of a running batch: some rows cross into a new block
        dict(name="tables_step", kind="tables", R=67, fresh=1, past=20000, block=64, stride=512,
             lens=3),
        # admission of a large wave of prompts into an empty pool
        dict(name="tables_prompts", kind="tables", R=4099, fresh=2500, past=0, block=32,
             stride=128, lens=4),
        # a small interactive batch over short windows: latency
        dict(name="decode_few", kind="decode", B=3, n_kv=2, G=4, hd=64, ctx=384, lo=20, hi=383,
             cap=30.0, window=256, slopes=False, docs=False, sinks=True, block=0, lens=5),
        # a serving batch with long histories, distance bias and packed documents
        dict(name="decode_long", kind="decode", B=33, n_kv=8, G=4, hd=128, ctx=16384, lo=1,
             hi=16383, cap=50.0, window=0, slopes=True, docs=True, sinks=False, block=0, lens=6),
        # a paged batch of wide heads with a sliding window and capped scores
        dict(name="decode_paged", kind="decode", B=47, n_kv=4, G=2, hd=256, ctx=8192, lo=100,
             hi=8191, cap=50.0, window=4096, slopes=False, docs=False, sinks=False, block=64,
             lens=7),
        # several documents packed into each prompt, with a distance bias
        dict(name="prefill_docs", kind="prefill", S=3, n_kv=8, G=4, hd=128, ctx=2048, fresh=2048,
             past=0, cap=0.0, window=0, slopes=True, docs=True, prefix=False, sinks=False,
             lens=8),
        # one more chunk of a long prompt whose head is a prefix attended both ways
        dict(name="prefill_chunk", kind="prefill", S=1, n_kv=8, G=8, hd=64, ctx=16384, fresh=517,
             past=15800, cap=40.0, window=0, slopes=False, docs=False, prefix=True, sinks=True,
             lens=9),
        # a few requests on one system prompt: latency
        dict(name="shared_few", kind="shared", B=6, groups=1, n_kv=2, G=4, hd=64, prefix=777,
             ctx=256, cap=0.0, slopes=False, sinks=True, lens=10),
        # two system prompts in one batch
        dict(name="shared_two", kind="shared", B=51, groups=2, n_kv=8, G=4, hd=128, prefix=8192,
             ctx=1024, cap=50.0, slopes=False, sinks=False, lens=11),
        # a large batch on one long document
        dict(name="shared_large", kind="shared", B=256, groups=1, n_kv=8, G=4, hd=128,
             prefix=32700, ctx=1024, cap=0.0, slopes=False, sinks=False, lens=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["map", "tables", "decode", "prefill", "shared"])
    lens = rng.randrange(1, 1 << 30)
    if kind == "map":
        R = _log_int(rng, 1, 800)
        return dict(kind=kind, R=R, fresh=_log_int(rng, 1, max(1, min(4096, 64000 // R))),
                    past=_log_int(rng, 1, 30000), lens=lens)
    if kind == "tables":
        return dict(kind=kind, R=_log_int(rng, 1, 4000), fresh=_log_int(rng, 1, 1200),
                    past=rng.choice([0, _log_int(rng, 1, 1500)]),
                    block=rng.choice([16, 32, 64, 128]), stride=256, lens=lens)
    hd = rng.choice([64, 128]) if kind != "decode" else rng.choice([64, 128, 256])
    G, n_kv = rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), rng.choice([1, 2, 3, 4, 8])
    cap = rng.choice([0.0, 30.0, 50.0])
    slopes = rng.random() < 0.5
    sinks = rng.random() < 0.4
    if kind == "decode":
        ctx, block = _log_int(rng, 128, 8192) // 128 * 128, rng.choice([0, 0, 64, 128])
        B = _log_int(rng, 1, max(1, min(64, 200_000_000 // (ctx * n_kv * hd))))
        return dict(kind=kind, B=B, n_kv=n_kv, G=G, hd=hd, ctx=ctx, lo=0, hi=ctx - 1, cap=cap,
                    window=rng.choice([0, _log_int(rng, 1, ctx)]), slopes=slopes,
                    docs=rng.random() < 0.5, sinks=sinks, block=block, lens=lens)
    if kind == "prefill":
        S = rng.choice([1, 2, 3, 5])
        fresh, past = _log_int(rng, 1, 1500 // S), rng.choice([0, _log_int(rng, 1, 4000)])
        return dict(kind=kind, S=S, n_kv=min(n_kv, 4), G=G, hd=hd, ctx=past + fresh + 37,
                    fresh=fresh, past=past, cap=cap,
                    window=rng.choice([0, _log_int(rng, 1, past + fresh)]), slopes=slopes,
                    docs=rng.random() < 0.5, prefix=rng.random() < 0.4, sinks=sinks, lens=lens)
    return dict(kind=kind, B=_log_int(rng, 2, 128), groups=rng.choice([1, 1, 2, 3]), n_kv=n_kv,
                G=G, hd=hd, prefix=_log_int(rng, 40, 16000), ctx=_log_int(rng, 8, 700), cap=cap,
                slopes=slopes, sinks=sinks, lens=lens)


# ------------------------------------------------------------------ lengths
# The lengths of a case (not its values) come from the case alone, so that its
# work is known without its inputs.
def _requests(case):
    r = random.Random(case["lens"])
    R, fresh, past = case["R"], case["fresh"], case["past"]
    f = [r.randint((fresh + 1) // 2, fresh) for _ in range(R)]
    p = [r.randint(0, past) for _ in range(R)]
    if case["kind"] == "map" and R > 3:
        f[1] = 0  # a request with nothing new in this step
    return p, f


def _decode_rows(case):
    r = random.Random(case["lens"])
    pos = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    pos[-1] = case["hi"]
    first = [r.randint(0, p) if r.random() < 0.5 else 0 for p in pos] if case["docs"] else None
    if first and case["B"] > 4:
        first[1] = pos[1] + 1  # a row whose mask leaves nothing
    lo = [max(first[b] if first else 0, p + 1 - case["window"] if case["window"] else 0, 0)
          for b, p in enumerate(pos)]
    return pos, first, lo


def _prefill_rows(case):
    """Per sequence (past, fresh); per token (sequence, position, document start, prefix end)."""
    r = random.Random(case["lens"])
    seqs, toks = [], []
    for s in range(case["S"]):
        n = case["fresh"] if s == 0 else r.randint((case["fresh"] + 1) // 2, case["fresh"])
        past = case["past"] if s == 0 else r.randint(case["past"] // 2, case["past"])
        seqs.append((past, n))
        total = past + n
        cuts = sorted({0, *(r.randrange(total) for _ in range(4))}) if case["docs"] else [0]
        end = r.randint(1, total) if case["prefix"] else 0
        if case["prefix"] and s == 0:
            end = past + n // 2 if n > 1 else total
        for p in range(past, total):
            doc = max(c for c in cuts if c <= p)
            toks.append((s, p, doc, end if p < end else 0))
    return seqs, toks


def _shared_rows(case):
    r = random.Random(case["lens"])
    B, n = case["B"], case["groups"]
    sizes = [max(1, B // n + (1 if g < B % n else 0)) for g in range(n)]
    sizes[-1] = max(0, B - sum(sizes[:-1]))
    plen = [case["prefix"] if g == 0 else r.randint(case["prefix"] // 2, case["prefix"])
            for g in range(n)]
    group = [g for g in range(n) for _ in range(sizes[g])][:B]
    own_pos = [r.randint(0, case["ctx"] - 1) for _ in range(B)]
    return group, plen, own_pos


# ------------------------------------------------------------------ work
def work(case):
    kind = case["kind"]
    if kind == "map":
        p, f = _requests(case)
        return {"bytes": 4 * (3 * len(f) + len(f) + 1 + 2 * sum(f)), "flops": sum(f)}
    if kind == "tables":
        p, f = _requests(case)
        bs = case["block"]
        need = sum(-(-(a + b) // bs) + (-a // bs) for a, b in zip(p, f))
        return {"bytes": 4 * (2 * len(f) + 2 * need + 2), "flops": len(f)}
    n_kv, G, hd = case["n_kv"], case["G"], case["hd"]
    n_head = n_kv * G
    kv = 2 * n_kv * hd * 4  # K and V of one key
    if kind == "decode":
        pos, first, lo = _decode_rows(case)
        keys = sum(max(0, p + 1 - a) for p, a in zip(pos, lo))
        hist = sum(max(0, p - a) for p, a in zip(pos, lo))
        rows = case["B"]
    elif kind == "prefill":
        seqs, toks = _prefill_rows(case)
        keys, hist, rows = 0, 0, len(toks)
        lows = {}
        for s, p, doc, end in toks:
            lo = max(doc, p + 1 - case["window"] if case["window"] else 0)
            keys += max(p, end - 1) + 1 - lo
            lows[s] = min(lows.get(s, lo), lo)
        hist = sum(max(0, seqs[s][0] - lo) for s, lo in lows.items())
    else:
        group, plen, own_pos = _shared_rows(case)
        rows = case["B"]
        keys = sum(plen[g] + o + 1 for g, o in zip(group, own_pos))
        hist = sum(plen[g] for g in set(group)) + sum(own_pos)
    return {"bytes": hist * kv + rows * (2 * n_head * hd * 4 + 2 * kv),
            "flops": 4 * hd * n_head * keys}


# ------------------------------------------------------------------ inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _i64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _model(case, rows, g):
    """One attention layer's parameters and a step's new vectors."""
    n_kv, hd = case["n_kv"], case["hd"]
    n_head = n_kv * case["G"]

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    i = torch.arange(hd // 2, device=DEV, dtype=torch.float64)
    st = {
        "q": rnd(rows, n_head, hd), "k_new": rnd(rows, n_kv, hd), "v_new": rnd(rows, n_kv, hd),
        "q_norm_w": 1 + 0.1 * rnd(hd), "k_norm_w": 1 + 0.1 * rnd(hd),
        "inv_freq": (10000.0 ** (-2 * i / hd)).float(),
        "sinks": rnd(n_head) if case["sinks"] else None,
        "out": torch.zeros(rows, n_head, hd, device=DEV), "scale": hd ** -0.5,
        "cap": case["cap"], "window": case.get("window", 0),
        "slopes": (2.0 ** (-8.0 * (torch.arange(n_head, device=DEV, dtype=torch.float64) + 1)
                           / n_head)).float() if case["slopes"] else None,
    }
    return st


def _cache(n, ctx, n_kv, hd, g):
    shape = (n, ctx, n_kv, hd)
    return (torch.randn(*shape, generator=g, device=DEV),
            torch.randn(*shape, generator=g, device=DEV))


def prepare(case, seed):
    kind = case["kind"]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    if kind in ("map", "tables"):
        p, f = _requests(case)
        R = case["R"]
        st.update(past=_i32(p), fresh=_i32(f), n_tok=sum(f))
        if kind == "map":
            st["n_slots"], st["slot_ctx"] = R, case["past"] + case["fresh"] + 1
            st["slots"] = torch.randperm(R, generator=g, device=DEV).to(torch.int32)
            st["starts"] = torch.empty(R + 1, dtype=torch.int32, device=DEV)
            st["tok_slots"] = torch.empty(sum(f), dtype=torch.int32, device=DEV)
            st["tok_positions"] = torch.empty(sum(f), dtype=torch.int32, device=DEV)
        else:
            bs = case["block"]
            have = [-(-a // bs) for a in p]
            need = [-(-(a + b) // bs) - h for a, b, h in zip(p, f, have)]
            st["n_slots"], st["slot_ctx"] = sum(have) + sum(need) + 5, bs
            ids = torch.randperm(st["n_slots"], generator=g, device=DEV).to(torch.int32)
            tables = torch.zeros(R, case["stride"], dtype=torch.int32, device=DEV)
            col = torch.arange(case["stride"], device=DEV)
            tables[col < _i64(have)[:, None]] = ids[:sum(have)]
            st.update(tables=tables, free=ids[sum(have):].contiguous(), max_need=max(need),
                      head=torch.tensor([2], dtype=torch.int32, device=DEV),
                      head_out=torch.zeros(1, dtype=torch.int32, device=DEV))
        if own:
            st["kv"] = _handle(st["n_slots"], st["slot_ctx"], 1, 64, 1, 1)
        return st
    n_kv, G, hd = case["n_kv"], case["G"], case["hd"]
    n_head = n_kv * G
    if kind == "decode":
        pos, first, lo = _decode_rows(case)
        B, bs = case["B"], case["block"]
        st.update(_model(case, B, g))
        st["positions"] = _i32(pos)
        st["doc_start"] = _i32(first) if first else None
        st["max_keys"] = max(pos) + 1
        if bs:
            per = -(-case["ctx"] // bs)
            blocks = B * per
            st["K"], st["V"] = _cache(blocks, bs, n_kv, hd, g)
            st["tables"] = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32).view(B, per)
        else:
            st["K"], st["V"] = _cache(B + 1, case["ctx"], n_kv, hd, g)
            st["slots"] = torch.randperm(B + 1, generator=g, device=DEV)[:B].to(torch.int32)
        rows = B
    elif kind == "prefill":
        seqs, toks = _prefill_rows(case)
        S, n = case["S"], len(toks)
        st.update(_model(case, n, g))
        st["K"], st["V"] = _cache(S, case["ctx"], n_kv, hd, g)
        seq_slots = torch.randperm(S, generator=g, device=DEV)
        seq = _i64([t[0] for t in toks])
        st["slots"] = seq_slots[seq].to(torch.int32)
        st["positions"] = _i32([t[1] for t in toks])
        st["doc_start"] = _i32([t[2] for t in toks]) if case["docs"] else None
        st["prefix_end"] = _i32([t[3] for t in toks]) if case["prefix"] else None
        # where the padded batch of the plain form finds its tokens, and back
        st["seq_slots"], st["max_keys"] = seq_slots, max(a + b for a, b in seqs)
        longest = max(b for _, b in seqs)
        at, start = [], 0
        for _, b in seqs:
            at.append([start + min(i, b - 1) for i in range(longest)])
            start += b
        st["pad"] = _i64(at)
        st["unpad"] = _i64([s * longest + p - seqs[s][0] for s, p, _, _ in toks])
        rows = n
    else:
        group, plen, own_pos = _shared_rows(case)
        B, n = case["B"], case["groups"]
        st.update(_model(case, B, g))
        st["K"], st["V"] = _cache(B, case["ctx"], n_kv, hd, g)
        st["PK"], st["PV"] = _cache(n, case["prefix"], n_kv, hd, g)
        order = torch.randperm(n, generator=g, device=DEV)
        st["slots"] = torch.randperm(B, generator=g, device=DEV).to(torch.int32)
        st["prefix_slots"] = order[_i64(group)].to(torch.int32)
        st["prefix_lens"] = _i32([plen[x] for x in group])
        st["positions"] = _i32([plen[x] + o for x, o in zip(group, own_pos)])
        st["max_own"] = max(own_pos) + 1
        st["group_slots"] = order
        sizes = [group.count(x) for x in range(n)]
        at, start = [], 0
        for c in sizes:
            at.append([start + min(i, c - 1) if c else 0 for i in range(max(sizes))])
            start += c
        st["pad"] = _i64(at)
        begin = [sum(sizes[:x]) for x in range(n)]
        st["unpad"] = _i64([x * max(sizes) + b - begin[x] for b, x in enumerate(group)])
        rows = B
    if own:
        K = st["K"]
        st["kv"] = _handle(K.shape[0], K.shape[1], n_kv, hd, rows, n_head, K, st["V"])
        if kind == "shared":
            PK = st["PK"]
            st["prefix_kv"] = _handle(PK.shape[0], PK.shape[1], n_kv, hd, 1, n_head, PK, st["PV"])
        from sequence_slot_kv_gb300 import Scores
        st["scores"] = Scores(cap=st["cap"], window=st["window"], slopes=st["slopes"],
                              doc_start=st.get("doc_start"), prefix_end=st.get("prefix_end"))
    return st


def _handle(n_slots, slot_ctx, n_kv, hd, rows, n_head, K=None, V=None):
    from sequence_slot_kv_gb300 import SlotKV
    return SlotKV(n_slots, slot_ctx, n_kv, hd, max_rows=rows, max_n_head=n_head, k_buf=K, v_buf=V)


# ------------------------------------------------------------------ one pass
def run(st):
    kind = st["case"]["kind"]
    return (_own if own else _plain)[kind](st)


def _own_map(st):
    st["kv"].token_map(st["slots"], st["past"], st["fresh"], st["starts"], st["tok_slots"],
                       st["tok_positions"])
    return st["starts"], st["tok_slots"], st["tok_positions"]


def _own_tables(st):
    st["kv"].extend_tables(st["past"], st["fresh"], st["tables"], st["free"], st["head"],
                           st["head_out"])
    return st["tables"], st["head_out"]


def _step(st):
    return st["q"], st["k_new"], st["v_new"], st["positions"]


def _rest(st):
    return (st["q_norm_w"], st["k_norm_w"], st["inv_freq"], st["sinks"], st["scores"], st["out"],
            EPS, st["scale"])


def _own_decode(st):
    if "tables" in st:
        st["kv"].decode_batch_attn_paged_scored(*_step(st), st["tables"], *_rest(st))
    else:
        st["kv"].decode_batch_attn_scored(*_step(st), st["slots"], *_rest(st))
    return st["out"], st["K"], st["V"]


def _own_prefill(st):
    st["kv"].prefill_batch_attn_scored(*_step(st), st["slots"], *_rest(st))
    return st["out"], st["K"], st["V"]


def _own_shared(st):
    st["kv"].decode_batch_attn_shared(*_step(st), st["slots"], st["prefix_kv"],
                                      st["prefix_slots"], st["prefix_lens"], *_rest(st))
    return st["out"], st["K"], st["V"]


_own = {"map": _own_map, "tables": _own_tables, "decode": _own_decode, "prefill": _own_prefill,
        "shared": _own_shared}


# ------------------------------------------------------------------ plain forms
def _plain_map(st):
    fresh, past = st["fresh"].long(), st["past"].long()
    starts = torch.cat([fresh.new_zeros(1), fresh.cumsum(0)])
    req = torch.repeat_interleave(fresh, output_size=st["n_tok"])
    pos = past[req] + torch.arange(st["n_tok"], device=DEV) - starts[req]
    return starts.int(), st["slots"][req], pos.int()


def _plain_tables(st):
    past, fresh, bs = st["past"].long(), st["fresh"].long(), st["slot_ctx"]
    have = (past + bs - 1) // bs
    need = (past + fresh + bs - 1) // bs - have
    ends = need.cumsum(0)
    head = st["head"].long()
    col = torch.arange(st["tables"].shape[1], device=DEV)[None, :] - have[:, None]
    new = (col >= 0) & (col < need[:, None])
    src = (head + (ends - need)[:, None] + col).clamp(0, st["free"].numel() - 1)
    st["tables"].copy_(torch.where(new, st["free"][src], st["tables"]))
    return st["tables"], (head + ends[-1]).int()


def _norm_rope(x, w, pos, inv_freq):
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    ang = pos.float()[:, None] * inv_freq  # the angle is the f32 product, by definition
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _vectors(st):
    """The step's queries [rows][n_kv][G][hd] (scaled), new keys and values."""
    q = _norm_rope(st["q"], st["q_norm_w"], st["positions"], st["inv_freq"]) * st["scale"]
    k = _norm_rope(st["k_new"], st["k_norm_w"], st["positions"], st["inv_freq"])
    n, n_head, hd = q.shape
    return q.view(n, k.shape[1], -1, hd), k, st["v_new"]


def _capped(st, s):
    return st["cap"] * torch.tanh(s / st["cap"]) if st["cap"] else s


def _weights(parts, sinks):
    """exp(s - m) of each part of the scores and the shared denominator, the sink logit in both."""
    m = torch.cat([p.amax(-1, keepdim=True) for p in parts], -1).amax(-1, keepdim=True)
    if sinks is not None:
        m = torch.maximum(m, sinks)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    es = [torch.exp(p - m) for p in parts]
    den = torch.cat([e.sum(-1, keepdim=True) for e in es], -1).sum(-1, keepdim=True)
    if sinks is not None:
        den = den + torch.exp(sinks - m)
    return es, torch.where(den == 0, torch.ones_like(den), den)


def _plain_decode(st):
    q, k, v = _vectors(st)
    B, n_kv, G, hd = q.shape
    pos, n = st["positions"].long(), st["max_keys"]
    t = torch.arange(n, device=DEV)
    row = torch.arange(B, device=DEV)
    if "tables" in st:
        bs = st["K"].shape[1]
        tab = st["tables"].long()
        st["K"][tab[row, pos // bs], pos % bs] = k
        st["V"][tab[row, pos // bs], pos % bs] = v
        used = tab[:, :-(-n // bs)]
        K = st["K"][used].flatten(1, 2)[:, :n]
        V = st["V"][used].flatten(1, 2)[:, :n]
    else:
        slots = st["slots"].long()
        st["K"][slots, pos] = k
        st["V"][slots, pos] = v
        K, V = st["K"][slots, :n], st["V"][slots, :n]
    s = torch.einsum("bkgd,btkd->bkgt", q, K)
    dist = pos[:, None] - t
    s = _capped(st, s)
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, n_kv, G, 1) * dist.float()[:, None, None]
    keep = dist >= 0
    if st["window"]:
        keep &= dist < st["window"]
    if st["doc_start"] is not None:
        keep &= t >= st["doc_start"].long()[:, None]
    s = s.masked_fill(~keep[:, None, None], -math.inf)
    sinks = None if st["sinks"] is None else st["sinks"].view(1, n_kv, G, 1)
    (e,), den = _weights([s], sinks)
    out = torch.einsum("bkgt,btkd->bkgd", e, V) / den
    return out.reshape(B, n_kv * G, hd), st["K"], st["V"]


def _plain_prefill(st):
    q, k, v = _vectors(st)
    n, n_kv, G, hd = q.shape
    pos, slots = st["positions"].long(), st["slots"].long()
    st["K"][slots, pos] = k
    st["V"][slots, pos] = v
    keys = st["max_keys"]
    K, V = st["K"][st["seq_slots"], :keys], st["V"][st["seq_slots"], :keys]
    pad, t = st["pad"], torch.arange(keys, device=DEV)
    s = torch.einsum("sikgd,stkd->skgit", q[pad], K)
    dist = pos[pad][:, :, None] - t
    s = _capped(st, s)
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, n_kv, G, 1, 1) * dist.abs().float()[:, None, None]
    last = pos if st["prefix_end"] is None else torch.maximum(pos, st["prefix_end"].long() - 1)
    keep = t <= last[pad][:, :, None]
    if st["window"]:
        keep &= dist < st["window"]
    if st["doc_start"] is not None:
        keep &= t >= st["doc_start"].long()[pad][:, :, None]
    s = s.masked_fill(~keep[:, None, None], -math.inf)
    sinks = None if st["sinks"] is None else st["sinks"].view(1, n_kv, G, 1, 1)
    (e,), den = _weights([s], sinks)
    out = torch.einsum("skgit,stkd->sikgd", e, V) / den.permute(0, 3, 1, 2, 4)
    return out.reshape(-1, n_kv * G, hd)[st["unpad"]], st["K"], st["V"]


def _plain_shared(st):
    q, k, v = _vectors(st)
    B, n_kv, G, hd = q.shape
    plen, slots = st["prefix_lens"].long(), st["slots"].long()
    own_pos = st["positions"].long() - plen
    st["K"][slots, own_pos] = k
    st["V"][slots, own_pos] = v
    # the rows of each prefix against its keys, once for all of them
    PK, PV = st["PK"][st["group_slots"]], st["PV"][st["group_slots"]]
    P = PK.shape[1]
    tp = torch.arange(P, device=DEV)
    s1 = torch.einsum("nikgd,ntkd->nikgt", q[st["pad"]], PK).flatten(0, 1)[st["unpad"]]
    # every row against its own keys
    n = st["max_own"]
    K, V = st["K"][slots, :n], st["V"][slots, :n]
    to = torch.arange(n, device=DEV)
    s2 = torch.einsum("bkgd,btkd->bkgt", q, K)
    d1, d2 = st["positions"].long()[:, None] - tp, own_pos[:, None] - to
    s1, s2 = _capped(st, s1), _capped(st, s2)
    if st["slopes"] is not None:
        sl = st["slopes"].view(1, n_kv, G, 1)
        s1 = s1 - sl * d1.float()[:, None, None]
        s2 = s2 - sl * d2.float()[:, None, None]
    s1 = s1.masked_fill((tp >= plen[:, None])[:, None, None], -math.inf)
    s2 = s2.masked_fill((d2 < 0)[:, None, None], -math.inf)
    sinks = None if st["sinks"] is None else st["sinks"].view(1, n_kv, G, 1)
    (e1, e2), den = _weights([s1, s2], sinks)
    o1 = torch.einsum("nikgt,ntkd->nikgd", e1[st["pad"]], PV).flatten(0, 1)[st["unpad"]]
    out = (o1 + torch.einsum("bkgt,btkd->bkgd", e2, V)) / den
    return out.reshape(B, n_kv * G, hd), st["K"], st["V"]


_plain = {"map": _plain_map, "tables": _plain_tables, "decode": _plain_decode,
          "prefill": _plain_prefill, "shared": _plain_shared}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "map":
        starts, slots, pos = [0], [], []
        for s, p, f in zip(st["slots"].tolist(), *_requests(case)):
            starts.append(starts[-1] + f)
            slots += [s] * f
            pos += range(p, p + f)
        return _i32(starts), _i32(slots), _i32(pos)
    if kind == "tables":
        bs, head = case["block"], int(st["head"])
        tables, free = st["tables"].cpu().numpy(), st["free"].cpu().numpy()
        for r, (p, f) in enumerate(zip(*_requests(case))):
            for i in range((p + bs - 1) // bs, (p + f + bs - 1) // bs):
                tables[r, i] = free[head]
                head += 1
        return torch.from_numpy(tables).to(DEV), _i32([head])
    n_kv, G, hd = case["n_kv"], case["G"], case["hd"]
    n = st["q"].shape[0]
    f64 = torch.float64
    half = hd // 2
    # RoPE rotates by the f32 product of position and frequency
    ang = (st["positions"].float()[:, None] * st["inv_freq"][None, :]).to(f64)

    def vec(x, w):
        x = x.to(f64)
        x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.to(f64)
        z = torch.complex(x[..., :half], x[..., half:])
        z = z * torch.polar(torch.ones_like(ang), ang)[:, None, :]
        return torch.cat([z.real, z.imag], -1)

    q, k = vec(st["q"], st["q_norm_w"]), vec(st["k_new"], st["k_norm_w"])
    K, V = st["K"].to(f64), st["V"].to(f64)
    pos = st["positions"].tolist()
    if kind == "shared":
        plen = st["prefix_lens"].tolist()
        at = [p - a for p, a in zip(pos, plen)]
    else:
        at = pos
    if "tables" in st:
        bs, tab = K.shape[1], st["tables"].long()
        where = [(int(tab[b, p // bs]), p % bs) for b, p in enumerate(pos)]
    else:
        where = list(zip(st["slots"].tolist(), at))
    for b, (x, y) in enumerate(where):
        K[x, y] = k[b]
        V[x, y] = st["v_new"][b].to(f64)
    slopes = torch.zeros(n_kv * G, device=DEV, dtype=f64) if st["slopes"] is None else st["slopes"].to(f64)

    def attend(rows, keys, values, p, t, keep):
        """Rows [r] against keys [m] of one sequence: p [r], t [m] positions, keep [r, m]."""
        out = torch.zeros(len(rows), n_kv * G, hd, device=DEV, dtype=f64)
        for h in range(n_kv * G):
            s = q[rows, h] @ keys[:, h // G].T * float(st["scale"])
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            s = s - slopes[h] * (p[:, None] - t[None, :]).abs()
            s = torch.where(keep, s, torch.full_like(s, -math.inf))
            if st["sinks"] is not None:
                col = st["sinks"][h].to(f64).expand(len(rows), 1)
                s = torch.cat([s, col], -1)
            w = torch.nan_to_num(torch.softmax(s, -1))  # a row without keys weighs nothing
            out[:, h] = w[:, :keys.shape[0]] @ values[:, h // G]
        return out

    res = torch.zeros(n, n_kv * G, hd, device=DEV, dtype=f64)
    if kind == "decode":
        _, _, lo = _decode_rows(case)
        for b, p in enumerate(pos):
            if lo[b] > p:
                continue
            t = torch.arange(lo[b], p + 1, device=DEV)
            if "tables" in st:
                sel = (tab[b, t // bs], t % bs)
            else:
                sel = (where[b][0], t)
            res[b] = attend([b], K[sel], V[sel], _i64([p]), t,
                            torch.ones(1, len(t), dtype=torch.bool, device=DEV))[0]
    elif kind == "prefill":
        _, toks = _prefill_rows(case)
        for s in range(case["S"]):
            rows = [i for i, x in enumerate(toks) if x[0] == s]
            p = _i64([toks[i][1] for i in rows])
            lo = [max(toks[i][2], toks[i][1] + 1 - case["window"] if case["window"] else 0)
                  for i in rows]
            hi = [max(toks[i][1], toks[i][3] - 1) for i in rows]
            t = torch.arange(max(hi) + 1, device=DEV)
            keep = (t >= _i64(lo)[:, None]) & (t <= _i64(hi)[:, None])
            slot = where[rows[0]][0]
            for c in range(0, len(rows), 512):  # a part of the rows at a time
                part = rows[c:c + 512]
                res[part] = attend(part, K[slot, :len(t)], V[slot, :len(t)], p[c:c + 512], t,
                                   keep[c:c + 512])
    else:
        PK, PV = st["PK"].to(f64), st["PV"].to(f64)
        for b in range(n):
            g, L, o = int(st["prefix_slots"][b]), plen[b], at[b]
            x = where[b][0]
            keys = torch.cat([PK[g, :L], K[x, :o + 1]])
            values = torch.cat([PV[g, :L], V[x, :o + 1]])
            t = torch.arange(L + o + 1, device=DEV)
            res[b] = attend([b], keys, values, _i64([pos[b]]), t,
                            torch.ones(1, len(t), dtype=torch.bool, device=DEV))[0]
    return res, K, V
