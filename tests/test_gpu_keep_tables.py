"""slot_kv_keep_path_paged on requests whose tables name blocks outside the pool."""
import pytest
import torch

import sequence_slot_kv_gb300 as skv
from test_gpu_pages import BAD, pool, u32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [1, 4, 32])
@pytest.mark.parametrize("bad", ["history", "far_history", "node", "last"])
@pytest.mark.parametrize("value", ["n_blocks", "all_ones"])
def test_any_used_entry_outside_the_pool(bs, bad, value):
    """A request that the tree call refuses moves nothing, wherever the entry is:
    in the history, under a node that is not kept, under the last node."""
    past, n, path = [40 * bs, 300 * bs], [9, 6 * bs], [[2, 5], [0, bs, bs + bs // 2]]
    path[1] = sorted(set(path[1]))
    per = 307
    N = 2 * per
    kv, K, V = pool(N, bs, 1, 64)
    tables = [list(range(per)), list(range(per, N))]
    at = {"history": 0, "far_history": 299, "node": 300 + 3, "last": 300 + 5}[bad]
    tables[1][at] = N if value == "n_blocks" else BAD
    tables[0][-1] = BAD  # behind the request's last node: not used
    wk, wv = K.clone(), V.clone()
    for k, j in enumerate(path[0]):
        s, d = past[0] + j, past[0] + k
        wk[d // bs, d % bs], wv[d // bs, d % bs] = K[s // bs, s % bs], V[s // bs, s % bs]
    flat = [x for p, m in zip(path, n) for x in p + [BAD] * (m - len(p))]
    kv.keep_path_paged(u32(sum(tables, [])).view(2, per), u32(past), u32([0, n[0], n[0] + n[1]]),
                       u32([len(p) for p in path]), u32(flat))
    assert torch.equal(K, wk) and torch.equal(V, wv)
    assert kv.get_status() == skv.DEV_RANGE
    kv.free()


def test_entries_behind_the_last_node_are_not_looked_at():
    kv, K, V = pool(8, 4, 1, 64)
    tables = u32([3, 5, BAD, 9]).view(1, 4)
    wk, wv = K.clone(), V.clone()
    wk[5, 1], wv[5, 1] = K[5, 3], V[5, 3]
    kv.keep_path_paged(tables, u32([5]), u32([0, 3]), u32([1]), u32([2, BAD, BAD]))
    assert torch.equal(K, wk) and torch.equal(V, wv)
    assert kv.get_status() == 0
    kv.free()
