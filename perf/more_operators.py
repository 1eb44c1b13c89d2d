"""The operators of speculative and branching decoding, as calls and in plain form.

Five operators that a serving loop makes beside the decode step, each with the
cases it is measured on:

  * ``tree``     attention of trees of drafted tokens over slots or a paged pool
                 (``tree_batch_attn``, ``tree_batch_attn_paged``);
  * ``keep``     the K and V rows of a verified tree's accepted path moved to
                 consecutive positions (``slot_kv_keep_path``,
                 ``slot_kv_keep_path_paged``);
  * ``fork``     block tables forked: full blocks shared, the partial one copied
                 (``slot_kv_fork_tables``);
  * ``free``     the blocks of finished or rolled-back requests given back to the
                 free list (``slot_kv_free_tables``);
  * ``compact``  a pool's blocks in use moved to its front, the block tables
                 rewritten (``slot_kv_compact_pool``).

With ``own`` false ``run`` is the plain form in elementary torch operations;
with ``own`` true it makes the framework's calls on the same state.  Arrays
that a call changes in place and that a scheduler hands in anew each time
(tables, share counts) are copied from their fresh values within the pass, on
both sides.
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
        # two interactive requests, each with a draft of a few tokens: latency
        dict(name="tree_chat", kind="tree", R=2, nodes=7, width=3, n_kv=2, G=4, hd=64, past=900,
             cap=0.0, window=0, slopes=False, docs=False, sinks=True, block=0, lens=1),
        # a serving batch verifying wide trees over ordinary histories
        dict(name="tree_serve", kind="tree", R=24, nodes=40, width=8, n_kv=8, G=4, hd=128,
             past=8000, cap=0.0, window=0, slopes=False, docs=False, sinks=False, block=0,
             lens=2),
        # wide heads with capped scores and a sliding window, over a paged pool
        dict(name="tree_window", kind="tree", R=12, nodes=27, width=1, n_kv=4, G=2, hd=256,
             past=9000, cap=50.0, window=4096, slopes=False, docs=True, sinks=False, block=64,
             lens=3),
        # a large paged batch, long histories, trees of up to 64 nodes, distance bias
        dict(name="tree_long", kind="tree", R=32, nodes=64, width=16, n_kv=8, G=5, hd=128,
             past=16000, cap=0.0, window=0, slopes=True, docs=False, sinks=True, block=128,
             lens=4),
        # the accepted rows of three verified drafts: latency
        dict(name="keep_few", kind="keep", R=3, nodes=16, n_kv=2, hd=64, past=700, block=0,
             lens=5),
        # and of a large paged batch
        dict(name="keep_batch", kind="keep", R=193, nodes=64, n_kv=8, hd=128, past=2000, block=64,
             lens=6),
        # two continuations of a prompt: latency
        dict(name="fork_few", kind="fork", rows=1, forks=2, n_kv=2, hd=64, past=500, block=64,
             lens=7),
        # several samples of each request of a batch
        dict(name="fork_samples", kind="fork", rows=96, forks=389, n_kv=8, hd=128, past=2500,
             block=64, lens=8),
        # a step's finished requests, some sharing a prompt's blocks
        dict(name="free_step", kind="free", R=7, past=3000, keep=False, block=32, shared=0.3,
             lens=9),
        # a wave of beams dropped or rolled back at once
        dict(name="free_wave", kind="free", R=1201, past=2400, keep=True, block=16, shared=0.5,
             lens=10),
        # a small pool tidied after a few requests have left
        dict(name="compact_few", kind="compact", R=3, past=300, blocks=41, n_kv=2, hd=64,
             block=64, shared=0.0, lens=11),
        # a large fragmented pool
        dict(name="compact_pool", kind="compact", R=61, past=2400, blocks=6007, n_kv=8, hd=128,
             block=32, shared=0.25, lens=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "keep", "fork", "free", "compact"])
    lens = rng.randrange(1, 1 << 30)
    if kind == "free":
        R = _log_int(rng, 1, 1200)
        return dict(kind=kind, R=R, past=_log_int(rng, 1, min(6000, 2_000_000 // R)),
                    keep=rng.random() < 0.5, block=rng.choice([16, 32, 64]),
                    shared=rng.choice([0.0, 0.3, 0.6]), lens=lens)
    hd, n_kv = rng.choice([64, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    if kind == "tree":
        G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        if hd == 256:
            n_kv = min(n_kv, 4)
        nodes = _log_int(rng, 1, 128)
        past = rng.choice([_log_int(rng, 1, 16000), _log_int(rng, 1, 16000), 0])
        # the largest listed case: 32 requests x 8 kv heads x 128 x 16000 keys x 5 x 64 rows
        most = 4_000_000_000 // ((past + nodes) * n_kv * hd * max(8, nodes * G // 8))
        return dict(kind=kind, R=_log_int(rng, 1, max(1, min(32, most * 4))), nodes=nodes,
                    width=rng.choice([1, 2, 4, 16]), n_kv=n_kv, G=G, hd=hd, past=past,
                    cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                    window=rng.choice([0, 0, _log_int(rng, 1, past + nodes)]),
                    slopes=rng.random() < 0.3, docs=rng.random() < 0.3,
                    sinks=rng.random() < 0.4, block=rng.choice([0, 64, 128]), lens=lens)
    if kind == "keep":
        return dict(kind=kind, R=_log_int(rng, 1, 190), nodes=_log_int(rng, 2, 100), n_kv=n_kv,
                    hd=min(hd, 128), past=_log_int(rng, 1, 2000), block=rng.choice([0, 32, 64]),
                    lens=lens)
    if kind == "fork":
        return dict(kind=kind, rows=_log_int(rng, 1, 90), forks=_log_int(rng, 1, 380), n_kv=n_kv,
                    hd=min(hd, 128), past=_log_int(rng, 1, 2500), block=rng.choice([32, 64]),
                    lens=lens)
    R, past, block = _log_int(rng, 1, 40), _log_int(rng, 1, 2400), rng.choice([16, 32])
    need = R * (past // block + 1)
    return dict(kind=kind, R=R, past=past, blocks=need + rng.randint(0, max(1, 4 * need // 5)),
                n_kv=n_kv, hd=min(hd, 128), block=block, shared=rng.choice([0.0, 0.25]),
                lens=lens)


# ------------------------------------------------------------------ lengths
# The lengths, trees and tables of a case (not its values) come from the case
# alone, so that its work is known without its inputs.
def _trees(case):
    """Per request its past and its nodes' parents (-1: the history's last key)."""
    r = random.Random(case["lens"])
    trees = []
    for i in range(case["R"]):
        n = r.randint((case["nodes"] + 1) // 2, case["nodes"])
        past = r.randint(case["past"] // 2, case["past"])
        if i == case["R"] - 1:
            n, past = case["nodes"], case["past"]
        # node 0 is the last accepted token, a child comes after its parent;
        # width 1: one chain
        trees.append((past, [-1] + [r.randint(max(0, j - case["width"]), j - 1)
                                    for j in range(1, n)]))
    return trees


def _docs(case):
    """Per request the first position of its document (0 without documents)."""
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, past) if case["docs"] and r.random() < 0.6 else 0
            for past, _ in _trees(case)]


def _paths(case):
    """Per request (past, nodes, kept path).  A kept node past the first ones is
    not among the first len(path), so a pass can be made again on its result."""
    r = random.Random(case["lens"])
    out = []
    for i in range(case["R"]):
        n = r.randint((case["nodes"] + 1) // 2, case["nodes"])
        past = r.randint(case["past"] // 2, case["past"])
        k = min(n, r.randint(1, 12))
        same = r.randint(1, k)  # the first nodes stay where they are
        rest = list(range(k, n))
        path = list(range(same)) + sorted(r.sample(rest, min(k - same, len(rest))))
        path = path if len(path) == k else list(range(len(path)))
        out.append((past, n, [] if i == 1 else path))  # (a request that keeps nothing)
    return out


def _fork_lens(case):
    """The rows' lengths, and each fork's source row."""
    r = random.Random(case["lens"])
    past = [r.randint((case["past"] + 1) // 2, case["past"]) for _ in range(case["rows"])]
    return past, [r.randrange(case["rows"]) for _ in range(case["forks"])]


def _held(case, n_blocks):
    """Per request its length and blocks, the blocks a permutation's first ones,
    some of them also another request's first ones; and the ids that are left."""
    r = random.Random(case["lens"])
    bs = case["block"]
    ids = list(range(n_blocks))
    r.shuffle(ids)
    rows, at = [], 0
    for _ in range(case["R"]):
        past = r.randint((case["past"] + 1) // 2, case["past"])
        nb = -(-past // bs)
        common = []
        if rows and r.random() < case["shared"]:
            other = rows[r.randrange(len(rows))][1]
            common = other[:r.randint(0, min(nb, len(other)))]
        rows.append((past, common + ids[at:at + nb - len(common)]))
        at += nb - len(common)
    return rows, ids[at:]


def _kept(case):
    r = random.Random(case["lens"] + 1)
    rows, _ = _held(case, _pool_blocks(case))
    return [r.randint(0, past) if case["keep"] and r.random() < 0.5 else 0 for past, _ in rows]


def _pool_blocks(case):
    return case["R"] * (-(-case["past"] // case["block"])) + 3


def work(case):
    kind = case["kind"]
    kv = 8 * case["n_kv"] * case["hd"] if "n_kv" in case else 0  # a position's K and V
    if kind == "tree":
        n_head, hd = case["n_kv"] * case["G"], case["hd"]
        hist = keys = rows = 0
        for (past, parents), doc in zip(_trees(case), _docs(case)):
            depth = []
            for a in parents:
                depth.append(0 if a < 0 else depth[a] + 1)
            lows = [max(doc, past + d + 1 - case["window"] if case["window"] else 0)
                    for d in depth]
            hist += max(0, past - min(lows))
            keys += sum(max(0, past - lo) + min(d + 1, max(0, past + d + 1 - lo))
                        for lo, d in zip(lows, depth))
            rows += len(parents)
        return {"bytes": hist * kv + rows * (2 * n_head * hd * 4 + 2 * kv),
                "flops": 4 * hd * n_head * keys}
    if kind == "keep":
        moved = sum(i != k for _, _, path in _paths(case) for k, i in enumerate(path))
        return {"bytes": 2 * moved * kv, "flops": 0}
    bs = case["block"]
    if kind == "fork":
        past, src = _fork_lens(case)
        entries = sum(past[s] // bs for s in src)
        return {"bytes": 2 * sum(past[s] % bs for s in src) * kv + 16 * entries, "flops": 0}
    if kind == "free":
        rows, _ = _held(case, _pool_blocks(case))
        entries = sum(len(ids) - -(-k // bs) for (_, ids), k in zip(rows, _kept(case)))
        return {"bytes": 16 * entries, "flops": 0}
    rows, _ = _held(case, case["blocks"])
    live = {i for _, ids in rows for i in ids}
    moved = sum(i >= len(live) for i in live)
    entries = sum(len(ids) for _, ids in rows)
    return {"bytes": 2 * moved * bs * kv + 8 * entries + 4 * (case["blocks"] - len(live)),
            "flops": 0}


# ------------------------------------------------------------------ inputs
def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _i64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


def _cache(n, ctx, n_kv, hd, g):
    shape = (n, ctx, n_kv, hd)
    return (torch.randn(*shape, generator=g, device=DEV),
            torch.randn(*shape, generator=g, device=DEV))


def _tables(rows, stride):
    """int32 [rows][stride] from lists of ids (entries past them are stale: 0)."""
    return _i32([list(x) + [0] * (stride - len(x)) for x in rows])


def _places(st, case, lens, g):
    """The K and V of requests that hold ``lens`` positions, with their slots or tables."""
    n_kv, hd, bs = case["n_kv"], case["hd"], case["block"]
    R = len(lens)
    if bs:
        per = -(-max(lens) // bs)
        st["K"], st["V"] = _cache(R * per, bs, n_kv, hd, g)
        st["tables"] = torch.randperm(R * per, generator=g, device=DEV).to(torch.int32).view(R, per)
    else:
        st["K"], st["V"] = _cache(R + 1, max(lens) + 5, n_kv, hd, g)
        st["slots"] = torch.randperm(R + 1, generator=g, device=DEV)[:R].to(torch.int32)


def prepare(case, seed):
    kind = case["kind"]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    rows, n_head = 1, case.get("n_kv", 1)
    if kind == "tree":
        trees = _trees(case)
        n_kv, hd = case["n_kv"], case["hd"]
        n_head = n_kv * case["G"]
        sizes = [len(par) for _, par in trees]
        rows = sum(sizes)
        i = torch.arange(hd // 2, device=DEV, dtype=torch.float64)
        slopes = 2.0 ** (-8.0 * (torch.arange(n_head, device=DEV, dtype=torch.float64) + 1) / n_head)
        st.update(q=rnd(rows, n_head, hd), k_new=rnd(rows, n_kv, hd), v_new=rnd(rows, n_kv, hd),
                  q_norm_w=1 + 0.1 * rnd(hd), k_norm_w=1 + 0.1 * rnd(hd),
                  inv_freq=(10000.0 ** (-2 * i / hd)).float(),
                  sinks=rnd(n_head) if case["sinks"] else None,
                  slopes=slopes.float() if case["slopes"] else None,
                  out=torch.zeros(rows, n_head, hd, device=DEV), scale=hd ** -0.5)
        _places(st, case, [past + n for (past, _), n in zip(trees, sizes)], g)
        starts = [sum(sizes[:r]) for r in range(len(sizes) + 1)]
        st.update(past=_i32([past for past, _ in trees]), starts=_i32(starts),
                  parents=_i32([a for _, par in trees for a in par]),
                  doc_start=_i32(_docs(case)) if case["docs"] else None, most=max(sizes),
                  max_keys=max(past + n for (past, _), n in zip(trees, sizes)))
    elif kind == "keep":
        paths = _paths(case)
        _places(st, case, [past + n for past, n, _ in paths], g)
        sizes = [n for _, n, _ in paths]
        st.update(past=_i32([past for past, _, _ in paths]),
                  starts=_i32([sum(sizes[:r]) for r in range(len(sizes) + 1)]),
                  n_keep=_i32([len(path) for _, _, path in paths]),
                  path=_i32([x for _, n, path in paths for x in path + [0] * (n - len(path))]),
                  most=max(len(path) for _, _, path in paths))
    elif kind == "fork":
        past, src = _fork_lens(case)
        bs = case["block"]
        held = [-(-p // bs) for p in past]
        n = sum(held) + len(src) + 3
        ids = torch.randperm(n, generator=g, device=DEV).tolist()
        at = [sum(held[:r]) for r in range(len(held) + 1)]
        stride = max(held) + 2
        st["K"], st["V"] = _cache(n, bs, case["n_kv"], case["hd"], g)
        st.update(past=_i32(past), src=_i32(src), head=_i32([1]), head_out=_i32([0]),
                  tables=_tables([ids[at[r]:at[r + 1]] for r in range(len(held))], stride),
                  out_tables=torch.zeros(len(src), stride, dtype=torch.int32, device=DEV),
                  free=_i32(ids[at[-1]:]), shares0=torch.zeros(n, dtype=torch.int32, device=DEV))
        st["shares"] = st["shares0"].clone()
    else:
        compact = kind == "compact"
        n = case["blocks"] if compact else _pool_blocks(case)
        held, left = _held(case, n)
        if not compact:  # (which of a pool's blocks move is the case's, with its work)
            name = torch.randperm(n, generator=g, device=DEV).tolist()
            held, left = [(past, [name[i] for i in ids]) for past, ids in held], [name[i] for i in left]
        count = torch.zeros(n, dtype=torch.int32)
        every = torch.tensor([i for _, ids in held for i in ids])
        count.index_add_(0, every, torch.ones(len(every), dtype=torch.int32))
        stride = max(len(ids) for _, ids in held) + 1
        # the free list as earlier steps leave it: what is before the head was taken
        st.update(past=_i32([past for past, _ in held]),
                  tables0=_tables([ids for _, ids in held], stride),
                  shares0=(count - 1).clamp(min=0).to(DEV),
                  free=_i32([0] * (n - len(left)) + left), head0=_i32([n - len(left)]),
                  head_out=_i32([0]))
        st.update(tables=st["tables0"].clone(), shares=st["shares0"].clone(),
                  head=st["head0"].clone())
        if compact:
            st["K"], st["V"] = _cache(n, case["block"], case["n_kv"], case["hd"], g)
        else:
            st["n_blocks"] = n
            st["keep"] = _i32(_kept(case)) if case["keep"] else None
    if own:
        from sequence_slot_kv_gb300 import Scores, SlotKV
        if kind == "free":  # the call reads no K or V: a pool of narrow rows
            st["kv"] = SlotKV(st["n_blocks"], case["block"], 1, 64, max_rows=1, max_n_head=1)
        else:
            K = st["K"]
            st["kv"] = SlotKV(K.shape[0], K.shape[1], case["n_kv"], case["hd"], max_rows=rows,
                              max_n_head=n_head, k_buf=K, v_buf=st["V"])
        if kind == "tree":
            st["scores"] = Scores(cap=case["cap"], window=case["window"], slopes=st["slopes"],
                                  doc_start=st["doc_start"])
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    kind = st["case"]["kind"]
    return (_own if own else _plain)[kind](st)


def _own_tree(st):
    rest = (st["past"], st["starts"], st["parents"], st["q_norm_w"], st["k_norm_w"],
            st["inv_freq"], st["sinks"], st["scores"], st["out"], EPS, st["scale"])
    if "tables" in st:
        st["kv"].tree_batch_attn_paged(st["q"], st["k_new"], st["v_new"], st["tables"], *rest)
    else:
        st["kv"].tree_batch_attn(st["q"], st["k_new"], st["v_new"], st["slots"], *rest)
    return st["out"], st["K"], st["V"]


def _own_keep(st):
    if "tables" in st:
        st["kv"].keep_path_paged(st["tables"], st["past"], st["starts"], st["n_keep"], st["path"])
    else:
        st["kv"].keep_path(st["slots"], st["past"], st["starts"], st["n_keep"], st["path"])
    return st["K"], st["V"]


def _own_fork(st):
    st["shares"].copy_(st["shares0"])
    st["kv"].fork_tables(st["src"], st["past"], st["tables"], st["out_tables"], st["shares"],
                         st["free"], st["head"], st["head_out"])
    return st["out_tables"], st["shares"], st["head_out"], st["K"], st["V"]


def _own_free(st):
    st["shares"].copy_(st["shares0"])
    st["kv"].free_tables(st["past"], st["tables"], st["shares"], st["free"], st["head"],
                         st["head_out"], keep=st["keep"])
    return st["shares"], st["free"], st["head_out"]


def _own_compact(st):
    for name in ("tables", "shares", "head"):
        st[name].copy_(st[name + "0"])
    st["kv"].compact_pool(st["past"], st["tables"], st["shares"], st["free"], st["head"])
    return st["tables"], st["shares"], st["free"], st["head"], st["K"], st["V"]


_own = {"tree": _own_tree, "keep": _own_keep, "fork": _own_fork, "free": _own_free,
        "compact": _own_compact}


# ------------------------------------------------------------------ plain forms
def _norm_rope(x, w, pos, inv_freq):
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    ang = pos.float()[:, None] * inv_freq  # the angle is the f32 product, by definition
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _at(st, req, pos):
    """Where position pos of request req is: the first two indexes of K and V."""
    if "tables" in st:
        bs = st["K"].shape[1]
        return st["tables"].long()[req, pos // bs], pos % bs
    return st["slots"].long()[req], pos


def _plain_tree(st):
    case = st["case"]
    n_kv, G, hd = case["n_kv"], case["G"], case["hd"]
    past, starts, N = st["past"].long(), st["starts"].long(), st["most"]
    n, R = st["q"].shape[0], past.numel()
    sizes = starts[1:] - starts[:-1]
    i = torch.arange(N, device=DEV)
    real = i < sizes[:, None]                               # [R, N] nodes of the padded trees
    at = (starts[:-1, None] + i).clamp(max=n - 1)           # their rows
    parent = st["parents"].long()[at].masked_fill(~real, -1)
    # who is an ancestor of whom, itself included: reachability by squaring
    up = (i[None, None, :] == parent[:, :, None]) | torch.eye(N, dtype=torch.bool, device=DEV)
    up = up.float()
    for _ in range(max(1, math.ceil(math.log2(N + 1)))):
        up = (torch.bmm(up, up) > 0).float()
    depth = up.sum(-1).long() - 1
    node_pos = past[:, None] + depth                        # [R, N]
    req = torch.repeat_interleave(torch.arange(R, device=DEV), sizes, output_size=n)
    idx = torch.arange(n, device=DEV) - starts[req]
    pos = node_pos[req, idx]
    q = _norm_rope(st["q"], st["q_norm_w"], pos, st["inv_freq"]) * st["scale"]
    k = _norm_rope(st["k_new"], st["k_norm_w"], pos, st["inv_freq"])
    x, y = _at(st, req, past[req] + idx)
    st["K"][x, y] = k
    st["V"][x, y] = st["v_new"]
    T = st["max_keys"]
    t = torch.arange(T, device=DEV)
    if "tables" in st:
        used = st["tables"].long()[:, :-(-T // st["K"].shape[1])]
        K, V = st["K"][used].flatten(1, 2)[:, :T], st["V"][used].flatten(1, 2)[:, :T]
    else:
        slots = st["slots"].long()
        K, V = st["K"][slots, :T], st["V"][slots, :T]
    s = torch.einsum("rikgd,rtkd->rkgit", q.view(n, n_kv, G, hd)[at], K)
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    # a key's node in its tree (before it: the history), and its position
    node = (t - past[:, None]).clamp(0, N - 1)
    in_tree = t >= past[:, None]
    key_pos = torch.where(in_tree, torch.gather(node_pos, 1, node), t)
    dist = node_pos[:, :, None] - key_pos[:, None, :]
    keep = torch.gather(up, 2, node[:, None, :].expand(R, N, T)) > 0
    keep = torch.where(in_tree[:, None, :], keep & (t < (past + sizes)[:, None])[:, None, :], True)
    if case["window"]:
        keep &= dist < case["window"]
    if st["doc_start"] is not None:
        keep &= (key_pos >= st["doc_start"].long()[:, None])[:, None, :]
    if st["slopes"] is not None:
        s = s - st["slopes"].view(1, n_kv, G, 1, 1) * dist.float()[:, None, None]
    s = s.masked_fill(~keep[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    if st["sinks"] is not None:
        sinks = st["sinks"].view(1, n_kv, G, 1, 1)
        m = torch.maximum(m, sinks)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(s - m)
    den = e.sum(-1, keepdim=True)
    if st["sinks"] is not None:
        den = den + torch.exp(sinks - m)
    den = torch.where(den == 0, torch.ones_like(den), den)
    out = torch.einsum("rkgit,rtkd->rikgd", e, V) / den.permute(0, 3, 1, 2, 4)
    return out.reshape(R, N, n_kv * G, hd)[req, idx], st["K"], st["V"]


def _plain_keep(st):
    past, n_keep = st["past"].long(), st["n_keep"].long()
    R = past.numel()
    k = torch.arange(st["most"], device=DEV).expand(R, -1)
    row = (st["starts"].long()[:-1, None] + k).clamp(max=st["path"].numel() - 1)
    src = torch.where(k < n_keep[:, None], st["path"].long()[row], k)  # the others stay
    req = torch.arange(R, device=DEV)[:, None].expand_as(k)
    keep = (k < n_keep[:, None]).nonzero(as_tuple=True)
    a, b = _at(st, req[keep], (past[:, None] + src)[keep])
    x, y = _at(st, req[keep], (past[:, None] + k)[keep])
    st["K"][x, y] = st["K"][a, b]
    st["V"][x, y] = st["V"][a, b]
    return st["K"], st["V"]


def _plain_fork(st):
    st["shares"].copy_(st["shares0"])
    bs, src = st["K"].shape[1], st["src"].long()
    length = st["past"].long()[src]
    full, rest = length // bs, length % bs
    head = st["head"].long()
    ends = (rest > 0).long().cumsum(0)
    old = st["tables"][src]
    col = torch.arange(old.shape[1], device=DEV)
    shared = col < full[:, None]
    new = st["free"][(head + ends - 1).clamp(min=0)]
    part = (col == full[:, None]) & (rest > 0)[:, None]
    table = torch.where(shared, old, torch.where(part, new[:, None], st["out_tables"]))
    st["out_tables"].copy_(table)
    st["shares"].index_add_(0, torch.where(shared, old, 0).flatten(), shared.flatten().int())
    i = (rest > 0).nonzero()[:, 0]
    a, b = old[i, full[i]].long(), new[i].long()
    copied = (torch.arange(bs, device=DEV) < rest[i, None])[:, :, None, None]
    for X in (st["K"], st["V"]):
        X[b] = torch.where(copied, X[a], X[b])
    return st["out_tables"], st["shares"], (head + ends[-1]).int(), st["K"], st["V"]


def _used(st):
    """Which entries of the tables hold a block, past the kept ones."""
    bs = st["case"]["block"]
    col = torch.arange(st["tables"].shape[1], device=DEV)
    used = col < ((st["past"].long() + bs - 1) // bs)[:, None]
    if st.get("keep") is not None:
        used &= col >= ((st["keep"].long() + bs - 1) // bs)[:, None]
    return used


def _plain_free(st):
    st["shares"].copy_(st["shares0"])
    n = st["shares"].numel()
    used = _used(st).flatten()
    ids = torch.where(used, st["tables"].flatten().long(), n)  # n: no entry
    at = torch.arange(ids.numel(), device=DEV)
    count = torch.zeros(n + 1, dtype=torch.int64, device=DEV).index_add_(0, ids, used.long())
    first = torch.full((n + 1,), ids.numel(), device=DEV).scatter_reduce_(0, ids, at, "amin")
    shares = torch.cat([st["shares"].long(), st["shares"].new_zeros(1).long()])
    dead = count > shares
    st["shares"].copy_((shares - count).clamp(min=0)[:n])
    gone = used & dead[ids] & (first[ids] == at)
    order = gone.long().cumsum(0)
    head = st["head"].long() - order[-1]
    place = torch.where(gone, head + order - 1, n)
    free = torch.cat([st["free"], st["free"].new_zeros(1)])
    free[place] = ids.int()
    st["free"].copy_(free[:n])
    return st["shares"], st["free"], head.int()


def _plain_compact(st):
    for name in ("tables", "shares", "head"):
        st[name].copy_(st[name + "0"])
    n = st["shares"].numel()
    used = _used(st)
    live = torch.zeros(n, dtype=torch.bool, device=DEV)
    live[st["tables"][used].long()] = True
    L = int(live.sum())
    src, dst = live[L:].nonzero()[:, 0] + L, (~live[:L]).nonzero()[:, 0]
    to = torch.arange(n, device=DEV, dtype=torch.int32)
    to[src] = dst.int()
    st["tables"].copy_(torch.where(used, to[st["tables"].long()], st["tables"]))
    for X in (st["K"], st["V"], st["shares"]):
        X[dst] = X[src]
    st["shares"][L:] = 0
    free = st["free"].numel() - (n - L)
    st["free"][free:] = torch.arange(L, n, device=DEV, dtype=torch.int32)
    st["head"].fill_(free)
    return st["tables"], st["shares"], st["free"], st["head"], st["K"], st["V"]


_plain = {"tree": _plain_tree, "keep": _plain_keep, "fork": _plain_fork, "free": _plain_free,
          "compact": _plain_compact}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "tree":
        return _exact_tree(case, st)
    return _loops(case, st)


def _exact_tree(case, st):
    f64 = torch.float64
    n_kv, G, hd = case["n_kv"], case["G"], case["hd"]
    half = hd // 2
    pos, depths = [], []
    for past, parents in _trees(case):
        depth = []
        for a in parents:
            depth.append(0 if a < 0 else depth[a] + 1)
        depths.append(depth)
        pos += [past + d for d in depth]
    # RoPE rotates by the f32 product of position and frequency
    ang = (_i64(pos).float()[:, None] * st["inv_freq"][None, :]).to(f64)

    def vec(x, w):
        x = x.to(f64)
        x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * w.to(f64)
        z = torch.complex(x[..., :half], x[..., half:])
        z = z * torch.polar(torch.ones_like(ang), ang)[:, None, :]
        return torch.cat([z.real, z.imag], -1)

    q, k, v = vec(st["q"], st["q_norm_w"]), vec(st["k_new"], st["k_norm_w"]), st["v_new"].to(f64)
    K, V = st["K"].to(f64), st["V"].to(f64)
    res = torch.zeros(*st["q"].shape, device=DEV, dtype=f64)
    at = 0
    for r, ((past, parents), depth, doc) in enumerate(zip(_trees(case), depths, _docs(case))):
        n = len(parents)
        t = torch.arange(past + n, device=DEV)
        where = (st["tables"][r].long()[t // K.shape[1]], t % K.shape[1]) if "tables" in st else \
            (int(st["slots"][r]), t)
        keys, values = K[where].clone(), V[where].clone()
        keys[past:], values[past:] = k[at:at + n], v[at:at + n]
        K[where], V[where] = keys, values
        row_pos = past + _i64(depth)
        key_pos = torch.cat([t[:past], row_pos])
        line = torch.zeros(n, past + n, dtype=torch.bool)
        for i, a in enumerate(parents):
            if a >= 0:
                line[i] = line[a]
            else:
                line[i, :past] = True
            line[i, past + i] = True
        keep = line.to(DEV) & (key_pos >= doc)
        dist = row_pos[:, None] - key_pos[None, :]
        if case["window"]:
            keep &= dist < case["window"]
        for h in range(n_kv * G):
            s = q[at:at + n, h] @ keys[:, h // G].T * float(st["scale"])
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if st["slopes"] is not None:
                s = s - st["slopes"][h].to(f64) * dist
            s = torch.where(keep, s, torch.full_like(s, -math.inf))
            if st["sinks"] is not None:
                s = torch.cat([s, st["sinks"][h].to(f64).expand(n, 1)], -1)
            w = torch.nan_to_num(torch.softmax(s, -1))  # a row without keys weighs nothing
            res[at:at + n, h] = w[:, :past + n] @ values[:, h // G]
        at += n
    return res, K, V


def _loops(case, st):
    """The moves and lists of the other operators, one after the other."""
    kind, bs = case["kind"], case["block"]
    if kind == "keep":
        for r, (past, _, path) in enumerate(_paths(case)):
            for k, i in enumerate(path):
                a, b = (past + i, past + k)
                if bs:
                    row = st["tables"][r].tolist()
                    a, b = (row[a // bs], a % bs), (row[b // bs], b % bs)
                else:
                    a, b = (int(st["slots"][r]), a), (int(st["slots"][r]), b)
                for X in (st["K"], st["V"]):
                    X[b] = X[a].clone()
        return st["K"], st["V"]
    free, head, shares = st["free"].tolist(), int(st["head"]), st["shares"].tolist()
    tables = st["tables"].tolist()
    if kind == "fork":
        past, src = _fork_lens(case)
        out = st["out_tables"].tolist()
        for i, s in enumerate(src):
            full, rest = divmod(past[s], bs)
            for e in range(full):
                out[i][e] = tables[s][e]
                shares[out[i][e]] += 1
            if rest:
                out[i][full] = free[head]
                head += 1
                for X in (st["K"], st["V"]):
                    X[out[i][full], :rest] = X[tables[s][full], :rest].clone()
        return _i32(out), _i32(shares), _i32([head]), st["K"], st["V"]
    if kind == "free":
        rows, _ = _held(case, len(shares))
        dead = {}  # in the order of their first entries
        entries = [i for row, (_, ids), k in zip(tables, rows, _kept(case))
                   for i in row[-(-k // bs):len(ids)]]
        for i in entries:
            dead.setdefault(i, 0)
            dead[i] += 1
        gone = [i for i, c in dead.items() if c > shares[i]]
        for i, c in dead.items():
            shares[i] = max(0, shares[i] - c)
        free[head - len(gone):head] = gone
        return _i32(shares), _i32(free), _i32([head - len(gone)])
    rows, _ = _held(case, len(shares))
    live = sorted({i for _, ids in rows for i in ids})
    L = len(live)
    moves = dict(zip([i for i in live if i >= L], sorted(set(range(L)) - set(live))))
    for r, (_, ids) in enumerate(rows):
        tables[r][:len(ids)] = [moves.get(i, i) for i in ids]
    for a, b in moves.items():
        shares[b], shares[a] = shares[a], 0
        for X in (st["K"], st["V"]):
            X[b] = X[a]
    n = len(shares)
    free[len(free) - (n - L):] = range(L, n)
    return _i32(tables), _i32(shares), _i32(free), _i32([len(free) - (n - L)]), st["K"], st["V"]
