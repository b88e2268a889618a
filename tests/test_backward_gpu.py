"""attention_lse and attention_backward against 64-bit references (GPU)."""
import pytest
import torch

import masked_grouped_query_b200 as mgq
from tests import training_reference as ref

pytestmark = pytest.mark.gpu

CASES = [
    # (batch, q_len, kv_len, hq, hkv, d, causal, window, softcap, spread of q)
    (1, 1, 1, 1, 1, 128, True, None, None, 1),         # one row, one key
    (2, 1, 300, 8, 2, 128, True, None, None, 1),       # single-token rows of a group
    (1, 1, 2000, 32, 2, 64, True, 700, 30.0, 2),       # 16 rows, most keys outside the window
    (1, 128, 128, 2, 1, 128, True, None, None, 1),     # exactly one tile
    (1, 129, 257, 2, 2, 128, False, None, None, 1),    # one row and one key past a tile
    (1, 300, 300, 6, 2, 96, True, None, None, 2),      # ragged causal, groups of three
    (2, 200, 77, 4, 2, 72, True, None, None, 1),       # rows without a visible key
    (1, 260, 130, 4, 1, 80, True, 100, None, 1),       # the same with heads apart
    (1, 513, 900, 4, 1, 128, True, 128, 50.0, 3),      # window, softcap
    (1, 384, 384, 4, 4, 128, False, 65, 20.0, 6),      # window without causal, saturated cap
    (1, 700, 700, 8, 1, 32, True, 1, None, 1),         # the diagonal alone
    (3, 90, 90, 3, 3, 8, False, None, None, 4),        # the narrowest head
    (1, 512, 512, 2, 1, 128, True, None, None, 30),    # nearly one-hot probabilities
    (1, 333, 500, 4, 2, 256, True, 200, 30.0, 2),      # wide heads
    (2, 70, 65, 2, 1, 136, False, None, None, 1),      # just over 128 columns
    (1, 1000, 1000, 2, 1, 64, True, None, None, 1),    # several row and key tiles
    (2, 600, 2400, 16, 16, 128, True, 300, None, 1),   # more tiles than SMs, most keys hidden
    (2, 3000, 700, 8, 8, 96, True, None, 30.0, 2),     # more tiles than SMs, most rows empty
    (3, 290, 1200, 32, 16, 40, True, 64, None, 1),     # the same with one box of columns
]


def make(case, seed=0, dlse=False):
    b, lq, lk, hq, hkv, d, causal, window, cap, spread = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).bfloat16()

    t = dict(q=randn(b, hq, lq, d, s=spread), k=randn(b, hkv, lk, d), v=randn(b, hkv, lk, d),
             do=randn(b, hq, lq, d))
    t["dlse"] = torch.randn(b, hq, lq, generator=g, device="cuda") if dlse else None
    return t, dict(causal=causal, window=window, softcap=cap)


def paths(d):
    return (1, 2) if d <= 128 else (0,)


def forced(path, fn):
    mgq.set_override("force_path", path)
    try:
        r = fn()
        torch.cuda.synchronize()
        return r
    finally:
        mgq.set_override("force_path", 0)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_lse_forward(case):
    t, kw = make(case)
    f = ref.forward(t["q"], t["k"], t["v"], **kw)
    for path in paths(case[5]):
        o, lse = forced(path, lambda: mgq.attention_lse(t["q"], t["k"], t["v"], **kw))
        ref.assert_within("o", o, f["o"], ref.o_bound(f))
        empty = torch.isinf(f["lse"])
        assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
        assert (o[empty] == 0).all()
        zero = torch.zeros_like(f["lse"])
        ref.assert_within("lse", torch.where(empty, zero, lse.double()),
                          torch.where(empty, zero, f["lse"]), ref.lse_bound(f))
    assert mgq.status() & 0x1f == 0


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dlse", [False, True])
def test_backward(case, dlse):
    t, kw = make(case, seed=1, dlse=dlse)
    o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
    want, bound = ref.backward(t["q"], t["k"], t["v"], o, lse, t["do"], t["dlse"], **kw)
    for path in paths(case[5]):
        got = forced(path, lambda: mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse,
                                                          dlse=t["dlse"], **kw))
        for n, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
            ref.assert_within(f"{n} (path {path})", g, w, b)
    assert mgq.status() & 0x1f == 0
