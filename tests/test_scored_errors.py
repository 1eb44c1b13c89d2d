"""The call an error of the scored and shared steps names, without a GPU."""
import pytest
import torch

import sequence_slot_kv_gb300 as skv
from test_scored_args import _Handle


@pytest.mark.parametrize("compiled", [True, False])
def test_a_failing_call_is_named(compiled, monkeypatch):
    """A handle that is not allocated, with arguments that pass the checks."""
    h, i = _Handle(2, 64), torch.zeros(3, dtype=torch.int32)
    if compiled:
        class Compiled:
            def __getattr__(self, name):
                return lambda *a: 4  # SLOTKV_ERR_STATE

        monkeypatch.setattr(skv, "_call", Compiled())
    else:
        monkeypatch.setattr(skv, "_call", False)
        monkeypatch.setattr(skv, "_step_addrs", lambda *a: (3, 4, *[None] * 10, 0))
        monkeypatch.setattr(skv, "_int_addr", lambda *a: None)
    step = [torch.zeros(3, 4, 64)] * 3 + [i, i]
    rest = [None] * 5 + [torch.zeros(3, 4, 64), 1e-6, 0.1]
    for name, args in (("decode_batch_attn_scored", step + rest),
                       ("prefill_batch_attn_scored", step + rest),
                       ("decode_batch_attn_paged_scored", step[:4] + [torch.zeros(3, 1)] + rest),
                       ("decode_batch_attn_shared", step + [h, i, i] + rest)):
        with pytest.raises(skv.SlotKVError, match=name):
            getattr(h, name)(*args, stream=0)


def test_a_step_without_block_tables_is_refused(monkeypatch):
    monkeypatch.setattr(skv, "_call", False)
    h, i = _Handle(2, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_tables"):
        h.decode_batch_attn_paged_scored(torch.zeros(3, 4, 64), torch.zeros(3, 2, 64),
                                         torch.zeros(3, 2, 64), i, None, torch.ones(64),
                                         torch.ones(64), torch.ones(32), None, None,
                                         torch.zeros(3, 4, 64), 1e-6, 0.1)
