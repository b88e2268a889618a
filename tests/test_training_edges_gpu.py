"""The training operators where their formulas are easy to get wrong (GPU)."""
import math

import pytest
import torch

import masked_grouped_query_b200 as mgq
from tests import training_reference as ref
from tests.test_backward_gpu import forced, make

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- NaN and infinities
NAN_ROWS = [
    # (batch, q_len, kv_len, hq, hkv, d, causal, window, softcap, path)
    (4, 700, 700, 16, 16, 64, True, None, None, 2),       # tcgen05, not split
    (4, 700, 700, 16, 16, 64, True, None, 30.0, 2),
    (4, 700, 700, 16, 16, 128, True, None, 80.0, 2),
    (1, 300, 1500, 4, 2, 128, True, None, None, 2),       # split
    (1, 300, 1500, 4, 2, 128, True, None, 30.0, 2),
    (1, 300, 1500, 4, 2, 128, False, None, 80.0, 2),
    (1, 40, 3000, 2, 1, 128, True, None, None, 2),        # paired splits
    (1, 40, 3000, 2, 1, 128, True, None, 30.0, 2),
    (1, 40, 3000, 2, 1, 72, True, None, 80.0, 2),
    (1, 4, 3000, 2, 1, 128, True, None, None, 1),         # mma.sync, up to eight rows, split
    (16, 4, 100, 32, 16, 128, True, None, 30.0, 1),       # not split
    (1, 60, 3000, 2, 1, 64, True, None, None, 1),         # more rows, split
    (4, 700, 700, 16, 16, 256, True, 100, 30.0, 0),       # not split
]


def dims(case):
    return case[:9] + (1,), case[9]


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("case", NAN_ROWS, ids=str)
def test_rows_that_are_not_numbers(case, value):
    case, path = dims(case)
    t, kw = make(case, seed=26)
    o, lse = forced(path, lambda: mgq.attention_lse(t["q"], t["k"], t["v"], **kw))
    # A row of NaN, or an infinite logit without a softcap: the largest one less itself.
    row = case[1] // 2
    t["q"][0, 1, row, 3] = float(value)
    o2, lse2 = forced(path, lambda: mgq.attention_lse(t["q"], t["k"], t["v"], **kw))
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[0, 1, row] = True
    if kw["softcap"] is None:
        assert torch.equal(o[~hit], o2[~hit]) and torch.equal(lse[~hit], lse2[~hit])
    else:
        # Logits that are not finite leave the polynomial's range for their whole warp:
        # the other rows' tanh comes from the other formula, both within the bounds.
        clean = t["q"].clone()
        clean[0, 1, row, 3] = 0
        f = ref.forward(clean, t["k"], t["v"], **kw)
        for a, b, r in ((o, o2, ref.o_bound(f)), (lse, lse2, ref.lse_bound(f))):
            assert ((a[~hit].double() - b[~hit].double()).abs() <= 2 * r.expand(a.shape)[~hit]).all()
    if value == "nan" or kw["softcap"] is None:
        assert torch.isnan(lse2[hit]).all() and torch.isnan(o2[hit]).all()
    else:  # the cap makes them finite
        cap, kv = kw["softcap"], 1 // (case[3] // case[4])
        x = torch.tanh(t["k"][0, kv].double() @ t["q"][0, 1, row].double()) * cap
        x = x.masked_fill(~ref.visible(case[1], case[2], case[6], case[7], "cuda")[row], -math.inf)
        want = torch.logsumexp(x, 0).item()
        lim = cap * 4e-7 + ref.E32 * (1 + abs(want) + cap)
        assert abs(lse2[0, 1, row].item() - want) <= lim
        p, v = torch.softmax(x, 0), t["v"][0, kv].double()
        lim = (2 * ref.U16 + 2 * lim) * (p @ v.abs()) + 1e-30
        assert ((o2[0, 1, row].double() - p @ v).abs() <= lim).all()
    assert mgq.status() & 0x1f == 0
