"""Forks beside the rows they came from, and compaction over all of them."""
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
