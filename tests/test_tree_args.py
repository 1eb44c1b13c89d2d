"""What the tree calls and the calls on pages refuse, checked without a GPU:
every size, pointer and shape check that precedes a CUDA call."""
import ctypes

import pytest
import torch

import sequence_slot_kv_gb300 as skv

STATE = 4


def test_calls_on_no_handle():
    lib = skv._lib
    z = [None] * 12
    assert lib.tree_batch_attn(None, 1, 1, 2, *z[:11], None, None, 1e-6, 0.1, None) == STATE
    assert lib.tree_batch_attn_paged(None, 1, 1, 2, *z[:4], 1, *z[:7], None, None, 1e-6, 0.1,
                                     None) == STATE
    assert lib.slot_kv_keep_path(None, 1, 1, *z[:6]) == STATE
    assert lib.slot_kv_keep_path_paged(None, 1, 1, None, 1, *z[:5]) == STATE
    assert lib.slot_kv_fork_tables(None, 1, None, 1, None, None, 1, *z[:3], 1, *z[:3]) == STATE
    assert lib.slot_kv_free_tables(None, 1, *z[:3], 1, None, None, 1, *z[:3]) == STATE
    assert lib.slot_kv_compact_pool(None, 1, None, None, 1, None, None, 1, None, None) == STATE
    assert "handle" in skv.last_error()


class _Handle(skv.SlotKV):  # the geometry a SlotKV carries, without a device
    def __init__(self, n_kv, hd, n_slots=9):
        self.n_kv_head, self.head_dim, self.n_slots = n_kv, hd, n_slots
        self._h = ctypes.c_void_p()

    def free(self):
        pass


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def refused(call, good, name, bad, match=None, error=ValueError):
    with pytest.raises(error, match=match or name):
        call(**{**good, name: bad})


def test_tree_shapes():
    B, nh, nkv, hd, R = 5, 4, 2, 64, 3
    h = _Handle(nkv, hd)
    good = dict(q=torch.zeros(B, nh, hd), k_new=torch.zeros(B, nkv, hd),
                v_new=torch.zeros(B, nkv, hd), past=ints(R), starts=ints(R + 1), parents=ints(B),
                q_norm_w=torch.ones(hd), k_norm_w=torch.ones(hd), inv_freq=torch.ones(hd // 2),
                sinks=None, scores=None, out=torch.zeros(B, nh, hd), eps=1e-6, scale=0.1)
    for call, idx in ((h.tree_batch_attn, dict(slots=ints(R))),
                      (h.tree_batch_attn_paged, dict(block_tables=ints(R, 4)))):
        args = {**good, **idx}
        for name, bad in (("out", torch.zeros(B, nh + 1, hd)), ("k_new", torch.zeros(B, nkv, hd + 1)),
                          ("v_new", None), ("parents", ints(B - 1)), ("q_norm_w", torch.ones(hd - 1)),
                          ("past", None), ("starts", ints(R, 1)), ("parents", None),
                          ("q", torch.zeros(B, hd)), (next(iter(idx)), None)):
            refused(call, args, name, bad)
        refused(call, args, "past", [1, 2], error=TypeError)
        with pytest.raises(ValueError, match="CUDA"):
            call(**args)


def test_pages_shapes():
    h, R, n = _Handle(1, 64), 3, 9
    keep = dict(slots=ints(R), past=ints(R), starts=ints(R + 1), n_keep=ints(R), path=ints(7))
    for name, bad in (("past", None), ("path", ints(7, 1)), ("slots", None)):
        refused(h.keep_path, keep, name, bad)
    paged = {**{k: v for k, v in keep.items() if k != "slots"}, "block_tables": ints(R, 2)}
    refused(h.keep_path_paged, paged, "block_tables", ints(R))
    fork = dict(src=ints(2), past=ints(R), block_tables=ints(R, 4), out_tables=ints(2, 4),
                shares=ints(n), free_blocks=ints(5), head=ints(1))
    for name in fork:
        refused(h.fork_tables, fork, name, None)
    free = dict(past=ints(R), block_tables=ints(R, 4), shares=None, free_blocks=ints(5), head=ints(1))
    compact = dict(free)
    for call, good in ((h.free_tables, free), (h.compact_pool, compact)):
        for name in ("past", "block_tables", "free_blocks", "head"):
            refused(call, good, name, None)


@pytest.mark.gpu
def test_shapes_and_sizes_on_a_device():
    kv = skv.SlotKV(9, 48, 2, 64, 4, 4)
    R = 3

    def dev(t):
        return t.cuda()

    good = dict(q=torch.zeros(4, 4, 64).cuda(), k_new=torch.zeros(4, 2, 64).cuda(),
                v_new=torch.zeros(4, 2, 64).cuda(), slots=ints(R).cuda(), past=ints(R).cuda(),
                starts=ints(R + 1).cuda(), parents=ints(4).cuda(), q_norm_w=torch.ones(64).cuda(),
                k_norm_w=torch.ones(64).cuda(), inv_freq=torch.ones(32).cuda(), sinks=None,
                scores=None, out=torch.zeros(4, 4, 64).cuda(), eps=1e-6, scale=0.1)
    refused(kv.tree_batch_attn, good, "slots", dev(ints(R + 1)))
    refused(kv.tree_batch_attn, good, "starts", dev(ints(R)))
    refused(kv.tree_batch_attn, good, "parents", dev(ints(4)).long(), match="int32", error=TypeError)
    refused(kv.tree_batch_attn, good, "scores", skv.Scores(doc_start=dev(ints(4))), match="doc_start")
    refused(kv.tree_batch_attn, good, "scores", skv.Scores(prefix_end=dev(ints(R))),
            match="prefix_end", error=skv.SlotKVError)
    refused(kv.tree_batch_attn, good, "scores", skv.Scores(cap=-1.0), match="cap", error=skv.SlotKVError)
    refused(kv.tree_batch_attn, good, "q", torch.zeros(4, 64, 4).cuda().transpose(1, 2), match="contiguous")
    paged = {**{k: v for k, v in good.items() if k != "slots"}, "block_tables": dev(ints(R, 2))}
    # 48 positions are no whole number of 64-key tiles
    refused(kv.tree_batch_attn_paged, paged, "eps", 1e-6, match="multiple", error=skv.SlotKVError)
    # more rows or requests than the handle was allocated for
    many = {**good, "past": dev(ints(5)), "starts": dev(ints(6))}
    refused(kv.tree_batch_attn, many, "slots", dev(ints(5)), match="max_rows", error=skv.SlotKVError)
    keep = dict(slots=dev(ints(R)), past=dev(ints(R)), starts=dev(ints(R + 1)), n_keep=dev(ints(R)),
                path=dev(ints(4)))
    kv.keep_path(**{**keep, "path": dev(ints(5))})  # (no workspace, so not bound by max_rows)
    refused(kv.keep_path, keep, "n_keep", dev(ints(2)))
    free = dict(past=dev(ints(R)), block_tables=dev(ints(R, 4)), shares=None, free_blocks=dev(ints(5)),
                head=dev(ints(1)))
    for call in (kv.free_tables, kv.compact_pool):
        refused(call, free, "shares", dev(ints(8)))
        refused(call, free, "past", dev(ints(R + 1)))
        refused(call, free, "block_tables", dev(ints(R, 0)), match="bt_stride", error=skv.SlotKVError)
    refused(kv.free_tables, free, "keep", dev(ints(R - 1)))
    fork = dict(src=dev(ints(2)), past=dev(ints(R)), block_tables=dev(ints(R, 4)),
                out_tables=dev(ints(2, 4)), shares=dev(ints(9)), free_blocks=dev(ints(5)), head=dev(ints(1)))
    refused(kv.fork_tables, fork, "out_tables", dev(ints(2, 3)))
    refused(kv.fork_tables, fork, "shares", dev(ints(8)))
    assert kv.get_status() == 0
    kv.free()
