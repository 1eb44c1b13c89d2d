"""slot_kv_fork_tables with tens of thousands of forks."""
import random

import pytest
import torch

from test_gpu_pages import fork_case, pool, u32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("forks", [2047, 2048, 2049, 5000, 20011])
@pytest.mark.parametrize("same", [False, True])
def test_many_forks(forks, same):
    r = random.Random(forks + same)
    past = [0, 2, 4, 1, 3, 5, 8] + [r.randint(0, 9) for _ in range(20)]  # 9: more blocks than the table
    src = [r.randrange(len(past) + 1) for _ in range(forks)]              # the last one: no row
    fork_case(r, past, src, 2, 4, 1, 64, same=same)
    # a list that runs out somewhere in the middle
    fork_case(r, past, src, 2, 4, 1, 64, n_free=forks // 4, same=same)


def test_the_time_of_a_call_is_linear_in_the_forks():
    """16 times the forks take 16 times the time and less, not 256 times: below 64."""
    n, bs = 1 << 18, 4
    kv, _, _ = pool(8, bs, 1, 64)
    src, past = u32([0] * n), u32([8])
    tables, out = u32([3, 5]).view(1, 2), u32([0] * (2 * n)).view(n, 2)
    shares, free, head = u32([0] * 8), u32([7]), u32([0])

    def took(m):
        best = float("inf")
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            kv.fork_tables(src[:m], past, tables, out[:m], shares, free, head)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    few = took(n // 16)
    assert took(n) < 64 * few
    assert shares.tolist() == [0, 0, 0, 4 * (n + n // 16), 0, 4 * (n + n // 16), 0, 0]
    assert bool((out == tables).all()) and kv.get_status() == 0
    kv.free()


def test_many_forks_captured_and_replayed():
    """The call's two kernels in a graph, head advanced in place by every replay."""
    n, bs, blocks = 3000, 4, 3 * 1500 + 40
    kv, K, V = pool(blocks, bs, 1, 64)
    src, past = u32([i % 2 for i in range(n)]), u32([8, 6])
    tables, out = u32([3, 5, 9, 1]).view(2, 2), u32([0] * (2 * n)).view(n, 2)
    ids = [b for b in range(blocks) if b not in (3, 5, 9, 1)]
    shares, free, head = u32([0] * blocks), u32(ids), u32([0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.fork_tables(src, past, tables, out, shares, free, head)
    for i in range(3):
        g.replay()
        took = ids[1500 * i:1500 * (i + 1)]
        assert out[::2].tolist() == [[3, 5]] * 1500 and out[1::2].tolist() == [[9, b] for b in took]
        assert int(head) == 1500 * (i + 1)
        assert all(torch.equal(X[took, :2], X[1, :2].expand(1500, -1, -1, -1)) for X in (K, V))
    assert [int(shares[b]) for b in (3, 5, 9, 1)] == [4500, 4500, 4500, 0] and kv.get_status() == 0
    kv.free()
