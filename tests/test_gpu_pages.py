"""slot_kv_keep_path, slot_kv_fork_tables, slot_kv_free_tables and
slot_kv_compact_pool against plain loops: bits and whole numbers, so equal."""
import random

import pytest
import torch

import sequence_slot_kv_gb300 as skv
from sequence_slot_kv_gb300 import SlotKV
from tree64 import i32

pytestmark = pytest.mark.gpu
BAD = 0xFFFFFFFF


def signed(x):
    return [(v + 2 ** 31) % 2 ** 32 - 2 ** 31 for v in x]


def u32(x):
    return i32(signed(x))


def host(t):
    return [v % 2 ** 32 for v in t.flatten().tolist()]


def pool(n, bs, n_kv=2, hd=64, rows=512):
    kv = SlotKV(n, bs, n_kv, hd, rows, n_kv)
    K, V = kv.kv_tensors()
    K.copy_(torch.arange(K.numel(), device="cuda", dtype=torch.int32).view(torch.float32).view(K.shape))
    V.copy_(torch.arange(K.numel(), 2 * K.numel(), device="cuda", dtype=torch.int32).view(torch.float32).view(K.shape))
    return kv, K.view(torch.int32), V.view(torch.int32)


# ------------------------------------------------------------------ keep path
def keep_case(r, reqs, paged, bs, n_kv, hd):
    """reqs: (past, nodes, path).  Runs the call and checks every bit of K and V."""
    R = len(reqs)
    need = max([past + n for past, n, _ in reqs] + [1])
    if paged:
        per = -(-need // bs)
        kv, K, V = pool(R * per + 3, bs, n_kv, hd, 4096)
        ids = list(range(R * per + 3))
        r.shuffle(ids)
        tables = [ids[i * per:(i + 1) * per] for i in range(R)]
        row = lambda i, t: (tables[i][t // bs], t % bs)  # noqa: E731
    else:
        kv, K, V = pool(R + 1, need, n_kv, hd, 4096)
        slots = list(range(R + 1))
        r.shuffle(slots)
        row = lambda i, t: (slots[i], t)  # noqa: E731
    starts = [sum(n for _, n, _ in reqs[:i]) for i in range(R + 1)]
    path = [x for _, n, p in reqs for x in list(p) + [BAD] * (n - len(p))]
    args = (u32([p for p, _, _ in reqs]), u32(starts), u32([len(p) for _, _, p in reqs]), u32(path))
    wk, wv = K.clone(), V.clone()
    for i, (past, n, p) in enumerate(reqs):
        src = [row(i, past + j) for j in p]
        for k, s in enumerate(src):
            wk[row(i, past + k)], wv[row(i, past + k)] = K[s], V[s]
    if paged:
        kv.keep_path_paged(u32(sum(tables, [])).view(R, -1), *args)
    else:
        kv.keep_path(u32(slots[:R]), *args)
    assert torch.equal(K, wk) and torch.equal(V, wv)
    assert kv.get_status() == 0
    kv.free()


@pytest.mark.parametrize("paged,bs", [(False, 0), (True, 1), (True, 5), (True, 32)])
@pytest.mark.parametrize("n_kv,hd", [(1, 64), (8, 128), (3, 256)])
def test_keep_path(paged, bs, n_kv, hd):
    r = random.Random(bs + hd)
    reqs = []
    for n in (1, 2, 7, 8, 9, 33, 64, 250, 256, 3):
        for k in {0, 1, min(n, 5), n}:
            reqs.append((r.choice([0, 1, 31, 40]), n, sorted(r.sample(range(n), k))))
    keep_case(r, reqs, paged, bs, n_kv, hd)


@pytest.mark.parametrize("paged", [False, True])
def test_keep_path_overlaps(paged):
    """Rows that are the source of one move and the place of another: shifts by one
    and more, longer than a batch of loads."""
    r = random.Random(0)
    reqs = [(3, 256, list(range(s, 256))) for s in (0, 1, 2, 7, 8, 9, 100)]
    reqs.append((0, 256, list(range(0, 256, 2))))
    keep_case(r, reqs, paged, 16, 2, 64)


def test_keep_path_refused():
    """A path that is not increasing, leaves the tree, or a request out of range:
    nothing of it moves, the others do."""
    reqs = [(5, 6, [0, 2, 5]), (9, 4, [1, 3])]
    for kind in ("order", "twice", "far", "many", "slot", "long", "starts", "tree"):
        R, n = 2, 6
        kv, K, V = pool(3, 300, rows=1000)
        slots, past, starts, nk = [2, 0], [5, 9], [0, 6, 10], [3, 2]
        path = [0, 2, 5, 9, 9, 9, 1, 3, 9, 9]
        if kind == "order":
            path[6:8] = [3, 1]
        elif kind == "twice":
            path[6:8] = [2, 2]
        elif kind == "far":
            path[7] = 4
        elif kind == "many":
            nk[1] = 5
        elif kind == "slot":
            slots[1] = 3
        elif kind == "long":
            past[1] = 297
        elif kind == "starts":
            starts[2] = 11
        else:
            past[1], starts[2], path = 0, 6 + 257, path + [9] * 253
        wk, wv = K.clone(), V.clone()
        for k, i in enumerate(reqs[0][2]):
            wk[2, 5 + k], wv[2, 5 + k] = K[2, 5 + i], V[2, 5 + i]
        kv.keep_path(u32(slots), u32(past), u32(starts), u32(nk), u32(path))
        assert torch.equal(K, wk) and torch.equal(V, wv), kind
        assert kv.get_status() == skv.DEV_RANGE, kind
        kv.free()
    kv, K, V = pool(4, 8, rows=100)
    wk = K.clone()
    kv.keep_path_paged(u32([0, 4, 2, 3]).view(2, 2), u32([7, 7]), u32([0, 3, 6]), u32([2, 2]),
                       u32([0, 2, 0, 0, 2, 0]))
    wk[3, 0] = K[3, 1]  # request 1: place 8 takes place 9's row
    assert torch.equal(K, wk)
    assert kv.get_status() == skv.DEV_RANGE
    kv.free()


# ------------------------------------------------------------------ fork
def plain_fork(src, past, tables, out, shares, free, head, bs, n_blocks, K, V):
    tables, out, shares, K, V = [list(t) for t in tables], [list(t) for t in out], list(shares), K.clone(), V.clone()
    flag, stride = 0, len(out[0]) if out else 1
    for i, s in enumerate(src):
        if s >= len(past) or -(-past[s] // bs) > stride:
            flag = 1
            continue
        full, rest = divmod(past[s], bs)
        if rest and head >= len(free):
            flag = 1
            continue
        for e in range(full):
            out[i][e] = tables[s][e]
            if out[i][e] < n_blocks:
                shares[out[i][e]] += 1
            else:
                flag = 1
        if rest:
            new, old = free[head], tables[s][full]
            head += 1
            out[i][full] = new
            if new < n_blocks and old < n_blocks:
                K[new, :rest], V[new, :rest] = K[old, :rest], V[old, :rest]
            else:
                flag = 1
    return out, shares, head, K, V, flag


def fork_case(r, past, src, bs, stride, n_kv=2, hd=64, n_free=None, head=2, same=False, spoil=None):
    R = len(past)
    held = [min(stride, -(-p // bs)) for p in past]
    n = sum(held) + len(src) + head + 2
    kv, K, V = pool(n, bs, n_kv, hd)
    ids = list(range(n))
    r.shuffle(ids)
    tables, at = [], 0
    for h in held:
        tables.append(ids[at:at + h] + [BAD] * (stride - h))
        at += h
    free = ids[at:] if n_free is None else ids[at:at + n_free]
    out = [[r.randint(0, 1 << 30) for _ in range(stride)] for _ in src]
    shares = [r.randint(0, 3) for _ in range(n)]
    if spoil:
        spoil(tables, free, n)
    w = plain_fork(src, past, tables, out, shares, free, head, bs, n, K, V)
    ts, tf, th = u32(shares), u32(free), u32([head])
    tho = th if same else u32([77])
    tt, to = u32(sum(tables, [])).view(R, stride), u32(sum(out, [])).view(len(src), stride)
    kv.fork_tables(u32(src), u32(past), tt, to, ts, tf, th, tho)
    assert host(to) == sum(w[0], []) and host(ts) == w[1] and host(tho) == [w[2]]
    assert torch.equal(K, w[3]) and torch.equal(V, w[4])
    assert host(tt) == sum(tables, []) and host(tf) == free
    assert kv.get_status() == (skv.DEV_RANGE if w[5] else 0)
    kv.free()


@pytest.mark.parametrize("bs", [1, 7, 32])
@pytest.mark.parametrize("forks", [0, 1, 3, 255, 256, 257, 700])
@pytest.mark.parametrize("same", [False, True])
def test_fork_tables(bs, forks, same):
    r = random.Random(bs * forks + same)
    past = [0, 1, bs, bs - 1, bs + 1, 5 * bs, 5 * bs + bs // 2] + [r.randint(0, 6 * bs) for _ in range(9)]
    fork_case(r, past, [r.randrange(len(past)) for _ in range(forks)], bs, 7, same=same)


@pytest.mark.parametrize("n_kv,hd,bs", [(8, 128, 64), (3, 256, 16), (16, 256, 32)])
def test_fork_wide_rows(n_kv, hd, bs):
    r = random.Random(hd)
    past = [3 * bs + 1, 2 * bs - 1, bs // 2, 4 * bs]
    for forks in (1, 2, 40):
        fork_case(r, past, [r.randrange(4) for _ in range(forks)], bs, 5, n_kv, hd)


def test_fork_refused():
    r = random.Random(3)
    past = [10, 8, 33, 5, 0]
    fork_case(r, past, [0, 5, 1, 1 << 31, 3], 4, 9)                   # rows out of range
    fork_case(r, past, [0, 2, 3, 1, 2], 4, 8)                         # more blocks than the table has
    for n_free in range(2, 6):                                        # the free list runs out
        fork_case(r, past, [0, 1, 3, 0, 4, 1, 2], 4, 9, n_free=n_free)
        fork_case(r, past, [0, 1, 3, 0, 4, 1, 2], 4, 9, n_free=n_free, same=True)
    fork_case(r, past, [0, 3], 4, 9, n_free=1)                        # head behind its end

    def spoil(tables, free, n):
        tables[0][0], tables[3][1], free[3] = n, BAD, n + 5
    fork_case(r, past, [0, 3, 0, 1], 4, 9, spoil=spoil)               # ids outside the pool


def test_fork_overlap_is_refused():
    kv, _, _ = pool(8, 4)
    t = u32([0] * 12).view(4, 3)
    with pytest.raises(skv.SlotKVError, match="overlap"):
        kv.fork_tables(u32([0]), u32([3, 3]), t[:2], t[1:2], u32([0] * 8), u32([7]), u32([0]))
    kv.fork_tables(u32([0]), u32([3, 3]), t[:2], t[2:3], u32([0] * 8), u32([7]), u32([0]))
    assert host(t[2]) == [7, 0, 0] and kv.get_status() == 0
    kv.free()


# ------------------------------------------------------------------ free
def plain_free(past, keep, tables, shares, free, head, bs, n_blocks, stride):
    shares, free, flag = list(shares) if shares else None, list(free), 0
    if head > len(free):
        head, flag = len(free), 1
    order, times = [], {}
    for p, k, row in zip(past, keep, tables):
        if -(-p // bs) > stride:
            flag = 1
            continue
        for i in row[-(-k // bs):-(-p // bs)]:
            if i >= n_blocks:
                flag = 1
            elif shares is None:
                order.append(i)
            else:
                order += [i] if i not in times else []
                times[i] = times.get(i, 0) + 1
    if shares is not None:
        flag |= int(any(c > shares[i] + 1 for i, c in times.items()))
        order = [i for i in order if times[i] > shares[i]]
        for i, c in times.items():
            shares[i] = max(0, shares[i] - c)
    F = len(order)
    for k, i in enumerate(order):
        if head - F + k >= 0:
            free[head - F + k] = i
    return shares, free, max(0, head - F), flag | int(F > head)


def free_case(past, keep, tables, shares, free, head, bs, n, stride, same=False):
    kv, K, _ = pool(n, bs, 1, 64)
    k0 = K.clone()
    w = plain_free(past, keep or [0] * len(past), tables, shares, free, head, bs, n, stride)
    ts, tf, th = None if shares is None else u32(shares), u32(free), u32([head])
    tho = th if same else u32([5])
    tt = u32(sum(tables, [])).view(len(past), stride)
    kv.free_tables(u32(past), tt, ts, tf, th, tho, keep=None if keep is None else u32(keep))
    if shares is not None:
        assert host(ts) == w[0]
    assert host(tf) == w[1] and host(tho) == [w[2]]
    assert host(tt) == sum(tables, []) and torch.equal(K, k0)
    assert kv.get_status() == (skv.DEV_RANGE if w[3] else 0)
    kv.free()


def held_pool(r, R, bs, stride, shared):
    """Requests with blocks of a pool, some shared, and what is left of it."""
    n = R * stride + 5
    ids = list(range(n))
    r.shuffle(ids)
    past, tables, shares = [], [], [0] * n
    for i in range(R):
        p = r.choice([0, 1, bs, r.randint(0, stride * bs), stride * bs])
        nb = -(-p // bs)
        row = [ids.pop() for _ in range(nb)]
        if i and shared:
            j = r.randrange(i)
            m = r.randint(0, min(nb, -(-past[j] // bs)))
            for e in range(m):
                ids.append(row[e])
                row[e] = tables[j][e]
                shares[row[e]] += 1
        past.append(p)
        tables.append(row + [BAD] * (stride - nb))
    return n, past, tables, shares, ids


@pytest.mark.parametrize("R,stride", [(0, 1), (1, 1), (1, 200), (5, 33), (31, 32), (33, 31), (130, 65),
                                      (700, 40), (256, 33), (513, 32), (3000, 20), (40, 900)])
@pytest.mark.parametrize("shared", [None, False, True])
@pytest.mark.parametrize("same", [False, True])
def test_free_tables(R, stride, shared, same):
    r = random.Random(R * stride + bool(shared))
    bs = r.choice([1, 4, 16])
    n, past, tables, shares, left = held_pool(r, R, bs, stride, shared)
    free = [BAD] * (n - len(left)) + left
    for keep in (None, [r.choice([0, p, p // 2, p + 3, max(0, p - 1)]) for p in past]):
        free_case(past, keep, tables, None if shared is None else shares, free, n - len(left), bs, n,
                  stride, same)


def test_free_some_sharers():
    """Part of a block's sharers give it up; two entries of one row name a block."""
    tables = [[3, 4, 5], [3, 4, 6], [3, 7, 8], [9, 9, 1]]
    shares = [0, 0, 0, 2, 1, 0, 0, 0, 0, 1, 0, 0]
    for past in ([12, 0, 0, 0], [12, 12, 0, 0], [12, 12, 12, 0], [0, 0, 0, 8], [12, 12, 12, 12], [0, 5, 9, 1]):
        free_case(past, None, tables, shares, [BAD] * 12, 12, 4, 12, 3)


def test_free_refused():
    n = 12
    tables = [[3, 4, 5], [6, n, 7], [BAD, 8, 8]]
    shares = [0] * n
    free_case([12, 12, 0], None, tables, shares, [BAD] * n, n, 4, n, 3)    # an id outside the pool
    free_case([12, 12, 0], None, tables, None, [BAD] * n, n, 4, n, 3)
    free_case([13, 4, 0], None, tables, shares, [BAD] * n, n, 4, n, 3)     # more blocks than the table
    free_case([12, 0, 12], None, tables, shares, [BAD] * n, n, 4, n, 3)    # given up twice
    free_case([12, 4, 0], None, tables, shares, [BAD] * n, 2, 4, n, 3)     # no room
    free_case([12, 4, 0], None, tables, shares, [BAD] * n, 0, 4, n, 3)
    free_case([12, 4, 0], None, tables, shares, [BAD] * n, n + 9, 4, n, 3)  # head behind the list
    free_case([2 ** 32 - 1, 4, 0], None, tables, shares, [BAD] * n, n, 4, n, 3)


# ------------------------------------------------------------------ compact
def plain_compact(past, tables, shares, free, bs, n, stride, K, V):
    tables, shares, free = [list(t) for t in tables], list(shares) if shares else None, list(free)
    K, V, flag, used = K.clone(), V.clone(), 0, set()
    count = []
    for p, row in zip(past, tables):
        c = -(-p // bs)
        if c > stride:
            c, flag = stride, 1
        count.append(c)
        used |= {i for i in row[:c] if i < n}
        flag |= int(any(i >= n for i in row[:c]))
    L = len(used)
    to = dict(zip(sorted(i for i in used if i >= L), sorted(set(range(L)) - used)))
    for row, c in zip(tables, count):
        row[:c] = [to.get(i, i) for i in row[:c]]
    for a, b in to.items():
        K[b], V[b] = K[a], V[a]
        if shares:
            shares[b] = shares[a]
    if shares:
        shares[L:] = [0] * (n - L)
    F = min(n - L, len(free))
    free[len(free) - F:] = range(L, L + F)
    return tables, shares, free, len(free) - F, K, V, flag | int(F < n - L)


def compact_case(past, tables, shares, free, bs, n, stride, n_kv=1, hd=64):
    kv, K, V = pool(n, bs, n_kv, hd)
    w = plain_compact(past, tables, shares, free, bs, n, stride, K, V)
    ts, tf, th = None if shares is None else u32(shares), u32(free), u32([3])
    tt = u32(sum(tables, [])).view(len(past), stride)
    kv.compact_pool(u32(past), tt, ts, tf, th)
    assert host(tt) == sum(w[0], [])
    if shares is not None:
        assert host(ts) == w[1]
    assert host(tf) == w[2] and host(th) == [w[3]]
    assert torch.equal(K, w[4]) and torch.equal(V, w[5])
    assert kv.get_status() == (skv.DEV_RANGE if w[6] else 0)
    kv.compact_pool(u32(past), tt, ts, tf, th)  # nothing moves any more
    assert host(tt) == sum(w[0], []) and torch.equal(K, w[4]) and torch.equal(V, w[5])
    kv.free()


@pytest.mark.parametrize("R,stride,bs", [(0, 1, 4), (1, 1, 1), (1, 70, 8), (3, 11, 33), (33, 32, 2),
                                         (200, 40, 4), (820, 40, 1), (700, 95, 1)])
@pytest.mark.parametrize("shared", [None, False, True])
def test_compact_pool(R, stride, bs, shared):
    r = random.Random(R + stride)
    n, past, tables, shares, left = held_pool(r, R, bs, stride, shared)
    compact_case(past, tables, None if shared is None else shares, [BAD] * n, bs, n, stride)


def test_compact_ends():
    """Nothing in use, all in use, every block in use behind the free ones, and a pool of one."""
    n = 70
    compact_case([0, 0], [[BAD] * 35] * 2, [4] * n, [BAD] * n, 2, n, 35)
    ids = list(range(n))
    random.Random(1).shuffle(ids)
    compact_case([70, 70], [ids[:35], ids[35:]], list(range(n)), [BAD] * n, 2, n, 35)
    compact_case([70, 0], [list(range(69, 34, -1)), [BAD] * 35], list(range(n)), [BAD] * n, 2, n, 35)
    compact_case([1], [[0]], [0], [BAD], 2, 1, 1)
    compact_case([64, 1], [list(range(n - 32, n)) + [BAD] * 3, [31] + [BAD] * 34], [0] * n, [BAD] * n, 2, n, 35,
                 n_kv=8, hd=128)


def test_compact_refused():
    n = 12
    compact_case([12, 12], [[3, n, 5], [11, 7, BAD]], [0] * n, [BAD] * n, 4, n, 3)
    compact_case([13, 4], [[3, 9, 5], [11, 7, 1]], [0] * n, [BAD] * n, 4, n, 3)
    compact_case([12, 4], [[3, 9, 5], [11, 7, 1]], [0] * n, [BAD] * 5, 4, n, 3)
    compact_case([12, 4], [[3, 9, 5], [11, 7, 1]], [0] * n, [], 4, n, 3)


def test_pages_captured_and_replayed():
    """A beam step in a graph: fork two rows, free the old ones, roll back, compact."""
    bs, n = 4, 40
    kv, K, V = pool(n, bs)
    tables, out = u32([5, 6, 7, 0, 8, 9, 0, 0]).view(2, 4), u32([0] * 12).view(3, 4)
    shares, free, head = u32([0] * n), u32([BAD] * 6 + [i for i in range(n) if i not in (5, 6, 7, 8, 9)]), u32([6])
    src, past = u32([1, 1, 0]), u32([9, 6])
    new_past = u32([6, 6, 9])
    first = (K.clone(), V.clone(), tables.clone(), out.clone(), shares.clone(), free.clone(), head.clone())

    def step():
        kv.fork_tables(src, past, tables, out, shares, free, head)
        kv.free_tables(past, tables, shares, free, head)
        kv.free_tables(new_past, out, shares, free, head, keep=u32_keep)
        kv.compact_pool(u32_keep, out, shares, free, head)

    u32_keep = u32([4, 6, 5])
    step()
    want = [t.clone() for t in (K, V, tables, out, shares, free, head)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        for t, x in zip((K, V, tables, out, shares, free, head), first):
            t.copy_(x)
        g.replay()
        for t, x in zip((K, V, tables, out, shares, free, head), want):
            assert torch.equal(t, x)
    # 4 distinct blocks: 8 (shared by rows 0 and 1), row 1's copy, 5 and 6 of row 2
    assert host(head) == [len(free) - (n - 4)] and sorted(host(shares), reverse=True)[:2] == [1, 0]
    assert kv.get_status() == 0
    kv.free()


def test_compact_under_capture_needs_a_call_before():
    kv, _, _ = pool(4, 4)
    args = u32([1]), u32([3]).view(1, 1), None, u32([0] * 4), u32([0])
    with pytest.raises(skv.SlotKVError, match="before"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv.compact_pool(*args)
    kv.free()


def test_speculative_loop_over_pages():
    """Drafts verified, kept, extended, forked, freed and compacted together, against
    a cache that every request fills one token at a time."""
    from tree64 import Case, depths, line, tree
    r = random.Random(4)
    hd, n_kv, G, bs, n_blocks, stride = 128, 2, 2, 32, 64, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    R = 3
    kv = SlotKV(n_blocks, bs, n_kv, hd, 256, n_kv * G)
    w, inv = torch.ones(hd, device="cuda"), (1e4 ** (-2 * torch.arange(hd // 2, device="cuda").double() / hd)).float()
    tables, shares = u32([0] * (R * stride)).view(R, stride), u32([0] * n_blocks)
    free, head = u32(r.sample(range(n_blocks), n_blocks)), u32([0])
    past = [0] * R
    kept_k = [torch.empty(0, n_kv, hd, device="cuda") for _ in range(R)]  # what each cache must hold
    kept_v = [x.clone() for x in kept_k]
    for step in range(9):
        trees = [tree(r, r.randint(1, 20), 4) for _ in range(R)]
        n = [len(t) for t in trees]
        starts = [sum(n[:i]) for i in range(R + 1)]
        N = starts[-1]
        kv.extend_tables(u32(past), u32(n), tables, free, head)
        q, k, v = rnd(N, n_kv * G, hd), rnd(N, n_kv, hd), rnd(N, n_kv, hd)
        out = torch.zeros_like(q)
        kv.tree_batch_attn_paged(q, k, v, tables, u32(past), u32(starts), u32(sum(trees, [])), w, w, inv,
                                 None, None, out, 1e-6, hd ** -0.5)
        paths = []
        for t in trees:
            paths.append(line(t, r.randrange(len(t)))[::-1])
        # each accepted path's last node attends what a slot filled in order holds
        for i, (t, path) in enumerate(zip(trees, paths)):
            one = SlotKV(1, 400, n_kv, hd, 64, n_kv * G)
            K1, V1 = one.kv_tensors()
            K1[0, :past[i]], V1[0, :past[i]] = kept_k[i], kept_v[i]
            rows = [starts[i] + j for j in path]
            o = torch.empty(len(path), n_kv * G, hd, device="cuda")
            one.prefill_batch_attn(q[rows].contiguous(), k[rows].contiguous(), v[rows].contiguous(),
                                   u32(range(past[i], past[i] + len(path))), u32([0] * len(path)), w, w, inv,
                                   None, o, 1e-6, hd ** -0.5)
            assert float((out[rows] - o).abs().max()) < 1e-5
            kept_k[i] = K1[0, :past[i] + len(path)].clone()
            kept_v[i] = V1[0, :past[i] + len(path)].clone()
            one.free()
        flat = [x for t, path in zip(trees, paths) for x in path + [0] * (len(t) - len(path))]
        kv.keep_path_paged(tables, u32(past), u32(starts), u32([len(p) for p in paths]), u32(flat))
        grown = [a + b for a, b in zip(past, n)]
        past = [a + len(p) for a, p in zip(past, paths)]
        kv.free_tables(u32(grown), tables, shares, free, head, keep=u32(past))
        if step % 3 == 2:  # row 0 goes on as a fork of row 1, its own blocks freed
            new = u32([0] * (R * stride)).view(R, stride)
            kv.fork_tables(u32([1, 1, 2]), u32(past), tables, new, shares, free, head)
            kv.free_tables(u32(past), tables, shares, free, head)
            tables, past[0], kept_k[0], kept_v[0] = new, past[1], kept_k[1].clone(), kept_v[1].clone()
        if step % 4 == 3:
            kv.compact_pool(u32(past), tables, shares, free, head)
        K, V = kv.kv_tensors()
        for i in range(R):
            t = torch.arange(past[i], device="cuda")
            at = (tables[i].long()[t // bs], t % bs)
            assert torch.equal(K[at], kept_k[i]) and torch.equal(V[at], kept_v[i])
        # every block is in one place: held, or on the free list
        held = {tables[i, e].item() for i in range(R) for e in range(-(-past[i] // bs))}
        rest = host(free)[int(head):]
        assert len(set(rest)) == len(rest) and not held & set(rest) and len(held) + len(rest) == n_blocks
    assert kv.get_status() == 0
    kv.free()
