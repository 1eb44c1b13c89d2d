"""Trees of drafted tokens in 64 bits, row by row, from the definition
(include/slotkv.h, tree_batch_attn); the row itself is plain64's."""
import random

import torch

import plain64

F64 = torch.float64


def tree(rng, n, width, roots=1):
    """Parents of n nodes, the first ``roots`` of them following the history."""
    return [-1 if i < roots else rng.randint(max(0, i - width), i - 1) for i in range(n)]


def depths(parents):
    d = []
    for a in parents:
        d.append(0 if a < 0 else d[a] + 1)
    return d


def line(parents, i):
    """Node i and its ancestors."""
    nodes = []
    while i >= 0:
        nodes.append(i)
        i = parents[i]
    return nodes


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Requests [(past, parents)] on slots or on a shuffled pool, with values of a
    seed; ``pad`` rows belong to no request."""

    def __init__(self, reqs, n_kv, G, hd, block=0, seed=0, pad=0, sinks=False, slopes=False,
                 cap=0.0, window=0, docs=None, spare=7):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rng = random.Random(seed)

        def rnd(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.reqs, self.n_kv, self.G, self.hd, self.block = reqs, n_kv, G, hd, block
        self.n_head = n_kv * G
        R, n = len(reqs), sum(len(p) for _, p in reqs)
        self.rows = n
        B = n + pad
        self.q, self.k_new, self.v_new = rnd(B, self.n_head, hd), rnd(B, n_kv, hd), rnd(B, n_kv, hd)
        self.qw, self.kw = 1 + 0.1 * rnd(hd), 1 + 0.1 * rnd(hd)
        self.inv_freq = (10000.0 ** (-2 * torch.arange(hd // 2, device="cuda").double() / hd)).float()
        self.sinks = rnd(self.n_head) if sinks else None
        self.slopes = (2.0 ** (-8.0 * (torch.arange(self.n_head, device="cuda").double() + 1) /
                               self.n_head)).float() if slopes else None
        self.cap, self.window, self.docs = cap, window, docs
        self.scale, self.eps = hd ** -0.5, 1e-6
        longest = max([past + len(p) for past, p in reqs] + [1])
        if block:
            per = -(-longest // block)
            self.K, self.V = rnd(R * per + 2, block, n_kv, hd), rnd(R * per + 2, block, n_kv, hd)
            ids = list(range(R * per + 2))
            rng.shuffle(ids)
            self.tables = i32(ids[:R * per]).view(R, per)
        else:
            self.K, self.V = rnd(R + 1, longest + spare, n_kv, hd), rnd(R + 1, longest + spare, n_kv, hd)
            ids = list(range(R + 1))
            rng.shuffle(ids)
            self.slots = i32(ids[:R])
        self.past = i32([past for past, _ in reqs])
        self.starts = i32([sum(len(p) for _, p in reqs[:r]) for r in range(R + 1)])
        self.parents = i32([a for _, p in reqs for a in p] + [0] * pad)
        self.out = torch.full((B, self.n_head, hd), 7.5, device="cuda")

    def at(self, r, t):
        """Indexes of place(s) t of request r."""
        if self.block:
            return self.tables[r].long()[t // self.block], t % self.block
        return torch.full_like(t, int(self.slots[r])), t

    def handle(self):
        from sequence_slot_kv_gb300 import SlotKV
        return SlotKV(self.K.shape[0], self.K.shape[1], self.n_kv, self.hd,
                      max_rows=max(self.q.shape[0], len(self.reqs), 1), max_n_head=self.n_head,
                      k_buf=self.K, v_buf=self.V)

    def scores(self):
        from sequence_slot_kv_gb300 import Scores
        return Scores(cap=self.cap, window=self.window, slopes=self.slopes,
                      doc_start=None if self.docs is None else i32(self.docs))

    def run(self, kv, scores="own", stream=None):
        sc = self.scores() if scores == "own" else scores
        rest = (self.past, self.starts, self.parents, self.qw, self.kw, self.inv_freq, self.sinks,
                sc, self.out, self.eps, self.scale)
        if self.block:
            kv.tree_batch_attn_paged(self.q, self.k_new, self.v_new, self.tables, *rest,
                                     stream=stream)
        else:
            kv.tree_batch_attn(self.q, self.k_new, self.v_new, self.slots, *rest, stream=stream)
        return self.out

    def check(self, K0, V0, what="", vnorm=False, plus_one=False, skip=()):
        """out, K and V after a call against the definition; K0 and V0 were the
        cache's before it.  Requests in ``skip`` were refused.  Returns the others'
        outputs in 64 bits."""
        torch.cuda.synchronize()
        K, V = K0.clone(), V0.clone()
        row, exact = 0, []
        for r, (past, parents) in enumerate(self.reqs):
            n = len(parents)
            if n == 0:
                continue
            rows = slice(row, row + n)
            row += n
            if r in skip:
                assert bool((self.out[rows] == 7.5).all()), f"{what}: request {r} was written"
                continue
            dep = depths(parents)
            pos = i32([past + d for d in dep]).long()
            q = plain64.norm_rope(self.q[rows], self.qw, pos, self.inv_freq, self.eps, plus_one)
            k = plain64.norm_rope(self.k_new[rows], self.kw, pos, self.inv_freq, self.eps, plus_one)
            v = self.v_new[rows]
            if vnorm:
                v = v.double() / (v.double().pow(2).mean(-1, keepdim=True) + self.eps).sqrt()
            t = torch.arange(past + n, device="cuda")
            at = self.at(r, t)
            new = tuple(x[past:] for x in at)
            # k': a norm and a rotation in f32, a few ulp of the largest element each
            # (sum of squares 10, norm and weight 4, rotation 4: 18 roundings of 2^-24, twice)
            got = self.K[new].double()
            fine = torch.isfinite(k)
            assert torch.equal(torch.isfinite(got), fine), f"{what}: K of request {r}"
            tol = 2.0 ** -18 * torch.where(fine, k.abs(), 0.0).amax(-1, keepdim=True)
            assert bool(((got - k).abs()[fine] <= tol.expand_as(k)[fine]).all()), f"{what}: K of request {r}"
            if vnorm:
                assert float((self.V[new].double() - v).abs().max()) <= 2.0 ** -18 * float(v.abs().max())
            else:
                assert torch.equal(self.V[new].view(torch.int32), v.view(torch.int32)), f"{what}: V"
            K[new], V[new] = self.K[new], self.V[new]
            keys, values = K0[at].double(), V0[at].double()
            keys[past:], values[past:] = k, v.double()
            key_pos = torch.cat([t[:past], pos])
            want, tols = [], []
            for i in range(n):
                keep = torch.zeros(past + n, dtype=torch.bool)
                keep[:past] = True
                for j in line(parents, i):
                    keep[past + j] = True
                keep = keep.cuda()
                p = past + dep[i]
                if self.window:
                    keep &= p - key_pos < self.window
                if self.docs is not None:
                    keep &= key_pos >= self.docs[r]
                o, tol = plain64.row_attention(q[i], keys, values, p, key_pos, keep, self.scale,
                                               self.cap, self.slopes, self.sinks)
                want.append(o)
                tols.append(tol)
            plain64.check(self.out[rows], want, tols, f"{what} request {r}")
            exact += want
        assert bool((self.out[self.rows:] == 7.5).all()), f"{what}: rows of no request"
        assert torch.equal(self.K.view(torch.int32), K.view(torch.int32)), f"{what}: K elsewhere"
        assert torch.equal(self.V.view(torch.int32), V.view(torch.int32)), f"{what}: V elsewhere"
        return exact
