"""What the scored, shared and request-length calls refuse, checked without a
GPU: every size, pointer and shape check that precedes a CUDA call."""
import ctypes

import pytest
import torch

import sequence_slot_kv_gb300 as skv

ARG, STATE = 1, 4


def test_calls_on_no_handle():
    lib = skv._lib
    z = [None] * 9
    assert lib.decode_batch_attn_scored(None, 1, 2, *z, None, None, 1e-6, 0.1, None) == STATE
    assert lib.prefill_batch_attn_scored(None, 1, 2, *z, None, None, 1e-6, 0.1, None) == STATE
    assert lib.decode_batch_attn_paged_scored(None, 1, 2, *z[:5], 1, *z[:4], None, None, 1e-6, 0.1,
                                              None) == STATE
    assert lib.decode_batch_attn_shared(None, 1, 2, *z, *z[:3], None, None, 1e-6, 0.1,
                                        None) == STATE
    assert "handle" in skv.last_error()
    assert lib.slot_kv_token_map(None, 1, *z[:3], 1, *z[:4]) == STATE
    assert lib.slot_kv_extend_tables(None, 1, *z[:3], 1, None, 1, *z[:3]) == STATE


class _Handle(skv.SlotKV):  # the geometry a SlotKV carries, without a device
    def __init__(self, n_kv, hd):
        self.n_kv_head, self.head_dim, self._h = n_kv, hd, ctypes.c_void_p()

    def free(self):
        pass


def _step(B, nh, nkv, hd):
    i = torch.zeros(B, dtype=torch.int32)
    return dict(q=torch.zeros(B, nh, hd), k_new=torch.zeros(B, nkv, hd),
                v_new=torch.zeros(B, nkv, hd), positions=i, slots=i, q_norm_w=torch.ones(hd),
                k_norm_w=torch.ones(hd), inv_freq=torch.ones(hd // 2), sinks=None,
                out=torch.zeros(B, nh, hd), eps=1e-6, scale=0.1)


def test_binding_refuses_mismatched_shapes():
    B, nh, nkv, hd = 3, 8, 2, 64
    h, good = _Handle(nkv, hd), _step(3, 8, 2, 64)
    for call in (h.decode_batch_attn_scored, h.prefill_batch_attn_scored):
        for name, t in {"out": torch.zeros(B, nh - 1, hd), "k_new": torch.zeros(B, nkv + 1, hd),
                        "slots": torch.zeros(B - 1), "inv_freq": torch.ones(hd)}.items():
            with pytest.raises(ValueError, match=name):
                call(**{**good, name: t}, scores=None)
        with pytest.raises(ValueError, match="CUDA"):
            call(**good, scores=None)
    ok = torch.zeros(B, dtype=torch.int32)
    for bad in (dict(prefix_slots=ok[:2]), dict(prefix_lens=None)):
        with pytest.raises(ValueError, match=next(iter(bad))):
            h.decode_batch_attn_shared(**good, scores=None, prefix=h,
                                       **{"prefix_slots": ok, "prefix_lens": ok, **bad})
    with pytest.raises(TypeError, match="prefix"):
        h.decode_batch_attn_shared(**good, scores=None, prefix=3, prefix_slots=ok, prefix_lens=ok)
    paged = {k: v for k, v in good.items() if k != "slots"}
    with pytest.raises(ValueError, match="block_tables"):
        h.decode_batch_attn_paged_scored(**paged, block_tables=ok, scores=None)


def test_binding_refuses_scores():
    with pytest.raises(ValueError, match="CUDA"):
        skv.Scores(slopes=torch.zeros(4))
    with pytest.raises(ValueError, match="window"):
        skv.Scores(window=-1)
    with pytest.raises(ValueError, match="window"):
        skv.Scores(window=1 << 32)
    sc = skv.Scores(cap=2.0, window=9)
    assert sc.cap == 2.0 and sc.window == 9
    sc.doc_start, sc._arrays = torch.zeros(4, dtype=torch.int32), True
    with pytest.raises(ValueError, match="doc_start"):
        skv._scores(sc, 3, 8, 0)


def test_binding_refuses_request_arrays():
    h = _Handle(2, 64)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="fresh"):
        h.token_map(i, i, i[:2], torch.zeros(4), i, i)
    with pytest.raises(ValueError, match="starts"):
        h.token_map(i, i, i, i, i, i)
    with pytest.raises(ValueError, match="tok_positions"):
        h.token_map(i, i, i, torch.zeros(4), i, i[:2])
    with pytest.raises(ValueError, match="block_tables"):
        h.extend_tables(i, i, i, i, i[:1])
    with pytest.raises(ValueError, match="head"):
        h.extend_tables(i, i, torch.zeros(3, 4), i, i)
    with pytest.raises(ValueError, match="free_blocks"):
        h.extend_tables(i, i, torch.zeros(3, 4), torch.zeros(2, 2), i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        h.extend_tables(i, i, torch.zeros(3, 4, dtype=torch.int32), i, i[:1])
