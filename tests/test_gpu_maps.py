"""slot_kv_token_map and slot_kv_extend_tables against plain loops: whole
numbers, so equal to the last one."""
import numpy as np
import pytest
import torch

import sequence_slot_kv_gb300 as skv
from sequence_slot_kv_gb300 import SlotKV

pytestmark = pytest.mark.gpu
BAD = 0xFFFFFFFF


def dev(x):
    return torch.from_numpy(np.asarray(x, dtype=np.uint32).view(np.int32)).cuda()


def host(t):
    return t.cpu().numpy().view(np.uint32)


def plain_map(slots, past, fresh, n_slots, ctx, n_tok, keep):
    starts, ts, tp, flag, t = [0], list(keep[0]), list(keep[1]), 0, 0
    for s, p, f in zip(slots, past, fresh):
        ok = s < n_slots and p + f <= ctx
        flag |= int(f > 0 and not ok)
        for i in range(min(f, max(0, n_tok - t))):
            ts[t + i], tp[t + i] = (s if ok else BAD), (p + i) & BAD
        t += f
        starts.append(min(t, BAD))
    return starts, ts, tp, flag | int(t > n_tok)


@pytest.mark.parametrize("R,longest", [(0, 1), (1, 1), (1, 5000), (3, 700), (511, 3), (512, 9),
                                       (513, 40), (2000, 17), (1500, 1)])
@pytest.mark.parametrize("bad", [False, True])
def test_token_map(R, longest, bad):
    r = np.random.RandomState(R + longest + bad)
    n_slots, ctx = 64, 10000
    slots, past = r.randint(0, n_slots, R), r.randint(0, ctx - longest + 1, R)
    fresh = r.randint(0, longest + 1, R)
    if bad and R > 2:
        slots[R // 2], past[R - 1], fresh[R // 2], fresh[R - 1] = n_slots, ctx, 1, 1
    total = int(fresh.sum())
    kv = SlotKV(n_slots, ctx, 1, 64, 1, 1)
    for n_tok in {total, total + 37, max(0, total - 5)}:
        keep = r.randint(0, 1 << 30, n_tok), r.randint(0, 1 << 30, n_tok)
        ts, tp, starts = dev(keep[0]), dev(keep[1]), dev(np.zeros(R + 1))
        kv.token_map(dev(slots), dev(past), dev(fresh), starts, ts, tp)
        w = plain_map(slots.tolist(), past.tolist(), fresh.tolist(), n_slots, ctx, n_tok, keep)
        assert host(starts).tolist() == w[0]
        assert host(ts).tolist() == w[1] and host(tp).tolist() == w[2]
        assert kv.get_status() == (skv.DEV_RANGE if w[3] else 0)
    kv.free()


def test_token_map_lengths_past_32_bits():
    """Lengths whose sum passes 2^32: starts stop there, nothing is written out of place."""
    kv = SlotKV(4, 100, 1, 64, 1, 1)
    fresh = [3, 0xFFFFFFFF, 0xFFFFFFF0, 2]
    ts, tp, starts = dev([7] * 10), dev([7] * 10), dev([0] * 5)
    kv.token_map(dev([1, 2, 3, 0]), dev([5, 0, 0xFFFFFFFF, 0]), dev(fresh), starts, ts, tp)
    assert host(starts).tolist() == [0, 3, BAD, BAD, BAD]
    assert host(ts).tolist() == [1] * 3 + [BAD] * 7
    assert host(tp).tolist() == [5, 6, 7] + list(range(7))
    assert kv.get_status() == skv.DEV_RANGE
    kv.free()


def plain_tables(past, fresh, tables, free, head, bs):
    stride, flag, at, used = tables.shape[1], 0, head, head
    avail = max(head, len(free))
    for r, (p, f) in enumerate(zip(past, fresh)):
        have, want = -(-p // bs), -(-(p + f) // bs)
        if want > stride or p + f > BAD:
            flag = 1
            continue
        need = want - have
        if need and at + need > avail:
            flag = 1
        elif need:
            tables[r, have:want] = free[at:at + need]
            used = at + need
        at += need
    return tables, used, flag


@pytest.mark.parametrize("R,longest,bs,stride", [(0, 1, 64, 4), (1, 1, 64, 8), (1, 9000, 16, 700),
                                                 (67, 1, 64, 90), (513, 300, 32, 30),
                                                 (1100, 1, 16, 40), (700, 900, 16, 100)])
@pytest.mark.parametrize("short", [0, 1, 40])
def test_extend_tables(R, longest, bs, stride, short):
    r = np.random.RandomState(R + longest + short)
    past = r.randint(0, max(1, stride * bs - longest), R)
    past[:R // 4] = past[:R // 4] // bs * bs
    fresh = r.randint(0, longest + 1, R)
    if R > 3:
        past[2] = stride * bs - longest // 2  # passes its table, if it adds enough
    need = sum(-(-(p + f) // bs) + (-p // bs) for p, f in zip(past.tolist(), fresh.tolist())
               if -(-(p + f) // bs) <= stride)
    head0 = 3
    free = r.permutation(max(1, need + head0 + 11 - short * 12)) if short else r.permutation(need + head0)
    kv = SlotKV(8, bs, 1, 64, 1, 1)
    tab0 = r.randint(0, 1 << 30, (R, stride)).astype(np.uint32)
    for in_place in (False, True):
        tab, head, out = dev(tab0), dev([head0]), dev([99])
        kv.extend_tables(dev(past), dev(fresh), tab, dev(free), head, None if in_place else out)
        want, used, flag = plain_tables(past.tolist(), fresh.tolist(), tab0.copy(), free, head0, bs)
        assert np.array_equal(host(tab), want)
        assert int(host(head if in_place else out)[0]) == used
        assert in_place or int(host(head)[0]) == head0
        assert kv.get_status() == (skv.DEV_RANGE if flag else 0)
    kv.free()


def test_extend_tables_captured_steps():
    """A step's extension captured once and replayed: the head advances in place."""
    R, bs, stride, steps = 70, 16, 8, 100
    r = np.random.RandomState(1)
    past = r.randint(0, 20, R)
    kv = SlotKV(8, bs, 1, 64, 1, 1)
    pos, one, head = dev(past), dev(np.ones(R)), dev([0])
    free = r.permutation(R * stride)
    dfree = dev(free)
    tab = dev(np.full((R, stride), BAD))
    want, used = np.full((R, stride), BAD, dtype=np.uint32), 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.extend_tables(pos, one, tab, dfree, head)
        skv.slot_kv_advance_positions(pos, 1)
    for _ in range(steps):
        g.replay()
        want, used, flag = plain_tables(past.tolist(), [1] * R, want, free, used, bs)
        assert not flag
        past = past + 1
    torch.cuda.synchronize()
    assert np.array_equal(host(tab), want) and int(host(head)[0]) == used
    assert kv.get_status() == 0
    kv.free()
