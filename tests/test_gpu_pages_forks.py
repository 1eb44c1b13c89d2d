"""Forks beside the rows they came from: compaction over all of them, and a
roll-back into a block that a fork shares."""
import os
import random
import re

import pytest
import torch

from test_gpu_pages import host, pool, u32

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def rows_of(K, tables, past, bs):
    """Every row's keys, in order."""
    t = [torch.arange(p, device="cuda") for p in past]
    return [K[tables[r].long()[x // bs], x % bs].clone() for r, x in enumerate(t)]


def check_pool(tables, past, shares, free, head, n, bs):
    """Share counts are the entries beyond the first, and a block is held or free."""
    held = [int(tables[r, e]) for r, p in enumerate(past) for e in range(-(-p // bs))]
    assert host(shares) == [max(0, held.count(b) - 1) for b in range(n)]
    rest = host(free)[int(head):]
    assert sorted(rest + sorted(set(held))) == list(range(n))


@pytest.mark.parametrize("seed", range(4))
def test_forks_beside_their_source_are_compacted(seed):
    """One array holds the rows and, behind them, their forks: all of them are whole
    after a compaction that is given all of it."""
    r = random.Random(seed)
    bs, n, stride = 4, 64, 6
    kv, K, V = pool(n, bs)
    past = [r.randint(1, bs * stride) for _ in range(3)]
    src = [r.randrange(3) for _ in range(4)]
    ids = r.sample(range(n), n)
    every = u32([0] * (7 * stride)).view(7, stride)
    at = 0
    for i, p in enumerate(past):
        m = -(-p // bs)
        every[i, :m] = u32(ids[at:at + m])
        at += m
    shares, free, head = u32([0] * n), u32([0] * at + ids[at:]), u32([at])
    want = rows_of(K, every, past, bs), rows_of(V, every, past, bs)
    kv.fork_tables(u32(src), u32(past), every[:3], every[3:], shares, free, head)
    all_past = past + [past[s] for s in src]
    kv.compact_pool(u32(all_past), every, shares, free, head)
    for X, w in zip((K, V), want):
        got = rows_of(X, every, all_past, bs)
        assert all(torch.equal(got[i], w[i if i < 3 else src[i - 3]]) for i in range(7))
    assert kv.get_status() == 0
    check_pool(every, all_past, shares, free, head, n, bs)
    kv.free()


def test_the_readme_example_keeps_its_forks():
    """The calls on drafted trees and pages as README.md shows them, run as they stand."""
    with open(README) as f:
        code = re.search(r"Drafted trees and pages.*?```python\n(.*?)```", f.read(), re.S).group(1)
    bs, n, stride, hd, n_kv = 64, 24, 4, 64, 2
    kv, _, _ = pool(n, bs, n_kv, hd)
    K, V = kv.kv_tensors()
    K.normal_(), V.normal_()
    every = u32([0] * (4 * stride)).view(4, stride)
    every[0, :3], every[1, :2] = u32([20, 7, 23]), u32([22, 9])
    fresh = [3, 2]
    names = dict(
        torch=torch, pool=kv, hd=hd, tables=every[:2], out_tables=every[2:], all_tables=every,
        past=u32([150, 100]), starts=u32([0, 3, 5]), parents=u32([2 ** 32 - 1, 0, 1, 2 ** 32 - 1, 0]),
        q=torch.randn(5, n_kv, hd, device="cuda"), k_new=torch.randn(5, n_kv, hd, device="cuda"),
        v_new=torch.randn(5, n_kv, hd, device="cuda"), q_norm_w=torch.ones(hd, device="cuda"),
        k_norm_w=torch.ones(hd, device="cuda"), inv_freq=torch.ones(hd // 2, device="cuda"), sinks=None,
        rule=None, out=torch.empty(5, n_kv, hd, device="cuda"), n_keep=u32([3, 1]), path=u32([0, 1, 2, 0, 0]),
        grown=u32([150, 100]) + u32(fresh), shares=u32([0] * n), src=u32([0, 0]),
        free_blocks=u32([0] * 5 + [b for b in range(n) if b not in (20, 7, 23, 22, 9)]), head=u32([5]))
    exec(compile(code, "README.md", "exec"), names)
    past = [153, 101, 153, 153]
    assert names["past"].tolist() == past[:2]
    for X in (K, V):
        got = rows_of(X, every, past, bs)
        assert all(torch.equal(got[i], got[0]) for i in (2, 3))
    assert kv.get_status() == 0
    check_pool(every, past, names["shares"], names["free_blocks"], names["head"], n, bs)
    kv.free()


@pytest.mark.parametrize("length", [1, 63, 64, 65, 128, 150, 200, 230])
def test_a_row_rolled_back_into_a_shared_block_is_forked_first(length):
    """A row that goes back into a block that another row shares gets a copy of it
    by a fork, and only then goes on writing: the sharer keeps its bits."""
    bs, n, stride, n_kv, hd, past = 64, 32, 6, 2, 64, 230
    kv, K, V = pool(n, bs, n_kv, hd)
    Kf, Vf = kv.kv_tensors()
    Kf.normal_(), Vf.normal_()
    mine = [9, 30, 2, 17]
    every = u32([0] * (3 * stride)).view(3, stride)
    every[0, :4] = u32(mine)
    shares = u32([0] * n)
    free, head = u32([0] * 4 + [b for b in range(n) if b not in mine]), u32([4])
    kv.fork_tables(u32([0]), u32([past]), every[:1], every[1:2], shares, free, head)
    # row 1 back to `length` keys: its blocks behind go, the one that it ends in stays
    kv.free_tables(u32([past]), every[1:2], shares, free, head, keep=u32([length]))
    # so it is forked before it is written, and given up
    kv.fork_tables(u32([0]), u32([length]), every[1:2], every[2:], shares, free, head)
    kv.free_tables(u32([length]), every[1:2], shares, free, head)
    check_pool(every[[0, 2]], [past, length], shares, free, head, n, bs)
    first, keys = [X[mine].clone() for X in (K, V)], rows_of(K, every, [past], bs)[0]
    fresh = 70
    kv.extend_tables(u32([length]), u32([fresh]), every[2:], free, head)
    q, k, v = (torch.randn(fresh, h, hd, device="cuda") for h in (n_kv, n_kv, n_kv))
    w, f = torch.ones(hd, device="cuda"), torch.ones(hd // 2, device="cuda")
    kv.tree_batch_attn_paged(q, k, v, every[2:], u32([length]), u32([0, fresh]),
                             u32([2 ** 32 - 1] + list(range(fresh - 1))), w, w, f, None, None,
                             torch.empty_like(q), 1e-6, hd ** -0.5)
    assert all(torch.equal(X[mine], x) for X, x in zip((K, V), first))
    assert torch.equal(rows_of(K, every[2:], [length], bs)[0], keys[:length])
    got = rows_of(V, every[2:], [length + fresh], bs)[0]
    assert torch.equal(got[length:], v.view(torch.int32))
    check_pool(every[[0, 2]], [past, length + fresh], shares, free, head, n, bs)
    assert kv.get_status() == 0
    kv.free()
