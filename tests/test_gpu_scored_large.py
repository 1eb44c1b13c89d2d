"""The scored and shared calls in a cache whose offsets pass 32 bits, in
elements as well as in bytes: the last slot (or block), keys near its end."""
import pytest
import torch

from plain64 import F64, check, norm_rope, row_attention
from sequence_slot_kv_gb300 import Scores, SlotKV
from test_gpu_scored import EPS, Layer, i32

pytestmark = pytest.mark.gpu

N_KV, G, HD = 8, 2, 128


@pytest.fixture(scope="module")
def big():
    """70 slots of 65536 positions: 4.7e9 elements in K and in V (19 GB each)."""
    n_slots, ctx = 70, 65536
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough device memory")
    L = Layer(1, 16, N_KV, G, HD, 1, seed=3, slopes=True)
    L.kv.free()
    L.K = torch.empty(n_slots, ctx, N_KV, HD, device="cuda")
    L.V = torch.empty(n_slots, ctx, N_KV, HD, device="cuda")
    for x in (L.K, L.V):
        x[-1] = torch.randn(x.shape[1:], generator=L.g, device="cuda")
    yield L
    del L.K, L.V
    torch.cuda.empty_cache()


def expected(L, q, k, v, pos, keys, vals, window, cap=20.0):
    """keys[b], vals[b]: the row's keys from position first[b] = p + 1 - window on."""
    position = torch.tensor(pos, device="cuda")
    q64 = norm_rope(q, L.qw, position, L.inv, EPS)
    outs, tols = [], []
    for b, p in enumerate(pos):
        t = torch.arange(p + 1 - window, p + 1, device="cuda")
        o, tol = row_attention(q64[b], keys[b], vals[b], p, t, torch.ones_like(t, dtype=torch.bool),
                               L.scale, cap, L.slopes)
        outs.append(o)
        tols.append(tol)
    return outs, tols


def test_decode_and_prefill(big):
    L, ctx, W = big, 65536, 500
    kv = SlotKV(70, ctx, N_KV, HD, 64, N_KV * G, k_buf=L.K, v_buf=L.V)
    sc = Scores(20.0, W, L.slopes)
    for rows, name in ((1, "decode_batch_attn_scored"), (40, "prefill_batch_attn_scored")):
        pos = list(range(ctx - rows, ctx))
        q, k, v = L.step(rows)
        out = torch.empty(rows, N_KV * G, HD, device="cuda")
        getattr(kv, name)(q, k, v, i32(pos), i32([69] * rows), *L.params(), sc, out, EPS, L.scale)
        assert kv.get_status() == 0
        k64 = norm_rope(k, L.kw, torch.tensor(pos, device="cuda"), L.inv, EPS)
        got = L.K[69, pos].to(F64)
        assert float((got - k64).abs().max()) <= 2.0 ** -20 * float(k64.abs().max())
        assert torch.equal(L.V[69, pos], v)
        keys = [L.K[69, p + 1 - W:p + 1] for p in pos]
        vals = [L.V[69, p + 1 - W:p + 1] for p in pos]
        check(out, *expected(L, q, k, v, pos, keys, vals, W), name)
    kv.free()


def test_paged(big):
    L, W, bs = big, 300, 64
    n_blocks = 70 * 65536 // bs
    K, V = L.K.view(n_blocks, bs, N_KV, HD), L.V.view(n_blocks, bs, N_KV, HD)
    pool = SlotKV(n_blocks, bs, N_KV, HD, 1, N_KV * G, k_buf=K, v_buf=V)
    tab = [n_blocks - 1 - 3 * i for i in range(9)]  # from the last block down
    pos = [9 * bs - 5]
    q, k, v = L.step(1)
    out = torch.empty(1, N_KV * G, HD, device="cuda")
    pool.decode_batch_attn_paged_scored(q, k, v, i32(pos), i32([tab]), *L.params(),
                                        Scores(20.0, W, L.slopes), out, EPS, L.scale)
    assert pool.get_status() == 0
    t = torch.arange(pos[0] + 1 - W, pos[0] + 1, device="cuda")
    at = torch.tensor(tab, device="cuda")[t // bs], t % bs
    assert torch.equal(V[at][-1], v[0])
    check(out, *expected(L, q, k, v, pos, [K[at]], [V[at]], W), "paged")
    pool.free()


def test_shared(big):
    """The prefix in the last slot, as long as it is; the rows' own keys beside it."""
    L, ctx, W = big, 65536, 700
    pkv = SlotKV(70, ctx, N_KV, HD, 1, N_KV * G, k_buf=L.K, v_buf=L.V)
    K = L.rnd(3, 64, N_KV, HD)
    V = L.rnd(3, 64, N_KV, HD)
    kv = SlotKV(3, 64, N_KV, HD, 3, N_KV * G, k_buf=K, v_buf=V)
    own = [0, 63, 20]
    pos = [ctx + o for o in own]
    q, k, v = L.step(3)
    out = torch.empty(3, N_KV * G, HD, device="cuda")
    kv.decode_batch_attn_shared(q, k, v, i32(pos), i32([2, 0, 1]), pkv, i32([69] * 3), i32([ctx] * 3),
                                *L.params(), Scores(20.0, W, L.slopes), out, EPS, L.scale)
    assert kv.get_status() == 0
    keys, vals = [], []
    for s, o in zip([2, 0, 1], own):
        n = W - o - 1  # of the prefix
        keys.append(torch.cat([L.K[69, ctx - n:], K[s, :o + 1]]))
        vals.append(torch.cat([L.V[69, ctx - n:], V[s, :o + 1]]))
    check(out, *expected(L, q, k, v, pos, keys, vals, W), "shared")
    kv.free()
    pkv.free()
