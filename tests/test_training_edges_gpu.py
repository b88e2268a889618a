"""The training operators where their formulas are easy to get wrong (GPU)."""
import math
import warnings
from decimal import Decimal, getcontext

import pytest
import torch

import masked_grouped_query_b200 as mgq
from tests import training_reference as ref
from tests.test_backward_gpu import forced, make

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- statistics with large softcaps
ROW_MAX = [
    # (batch, q_len, kv_len, hq, hkv, d, causal, window, softcap, spread of q)
    (4, 700, 700, 16, 16, 64, True, None, 80.0, 1),        # not split; logits far below the cap
    (4, 700, 700, 16, 16, 64, True, None, 80.0, 60),       # logits past the cap
    (2, 640, 768, 32, 16, 128, False, None, 300.0, 30),    # not split, no mask
    (2, 640, 768, 32, 16, 128, True, 200, 300.0, 200),
    (1, 300, 500, 4, 2, 128, True, None, 80.0, 40),        # split
    (1, 300, 500, 4, 2, 40, False, None, 300.0, 150),
    (2, 200, 77, 4, 2, 72, True, None, 80.0, 20),          # rows without a visible key
    (1, 400, 130, 4, 1, 64, True, 100, 300.0, 100),
    (1, 40, 3000, 2, 1, 128, True, None, 80.0, 40),        # one row tile, paired splits
    (1, 1, 2000, 32, 2, 64, True, 700, 300.0, 100),
    (1, 333, 500, 4, 2, 256, True, 200, 300.0, 100),       # wide heads
]


def check_forward_and_gradients(case, kw, t, path):
    f = ref.forward(t["q"], t["k"], t["v"], **kw)
    o, lse = forced(path, lambda: mgq.attention_lse(t["q"], t["k"], t["v"], **kw))
    ref.assert_within("o", o, f["o"], ref.o_bound(f))
    empty = f["lse"] == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert (o[empty] == 0).all()
    zero = torch.zeros_like(f["lse"])
    ref.assert_within("lse", torch.where(empty, zero, lse.double()), torch.where(empty, zero, f["lse"]),
                      ref.lse_bound(f))
    want, bound = ref.backward(t["q"], t["k"], t["v"], o, lse, t["do"], None, **kw)
    got = forced(path, lambda: mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse, **kw))
    for n, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        ref.assert_within(n, g, w, b)
    assert mgq.status() & 0x1f == 0


@pytest.mark.parametrize("case,path", [(c, p) for c in ROW_MAX for p in ((0, 1, 2) if c[5] <= 128 else (0,))],
                         ids=str)
def test_row_max_softcap(case, path):
    # Caps above about 63.8 keep a running maximum.
    t, kw = make(case, seed=20)
    check_forward_and_gradients(case, kw, t, path)


@pytest.mark.parametrize("cap", [30.0, 50.0])
@pytest.mark.parametrize("case", [c for c in ROW_MAX if c[5] <= 128], ids=str)
def test_row_max_softcap_by_override(case, cap):
    t, kw = make(case, seed=21)
    kw["softcap"] = cap
    mgq.set_override("softcap_two_pass", 1)
    try:
        check_forward_and_gradients(case, kw, t, 2)
    finally:
        mgq.set_override("softcap_two_pass", 0)


# ---------------------------------------------------------------- rotary
def exact_turns(sections, theta, per_axis, positions):
    """Angles in turns, reduced to [0, 1): 96 bits of every frequency, whole-number products."""
    getcontext().prec = 60
    pi2, ln = Decimal("6.28318530717958647692528676655900576839433879875021164"), Decimal(theta).ln()
    out, i = [], 0
    for a, s in enumerate(sections):
        for j in range(s):
            f = (-ln * j / s if per_axis else -ln * i / sum(sections)).exp() / pi2
            f = int((f * 2 ** 96).to_integral_value())
            i += 1
            out.append([(p * f % 2 ** 96) / 2 ** 96 for p in positions[a]])
    return torch.tensor(out, dtype=torch.float64, device="cuda").T  # (length, pairs)


@pytest.mark.parametrize("theta", [0.01, 0.5, 1.0, 1.01, 1.5, 10.0, 100.0])
@pytest.mark.parametrize("sections,per_axis", [((32,), False), ((128,), False), ((61, 64), True)])
def test_rotary_frequencies_of_slow_decay(theta, sections, per_axis):
    # Positions near 2^31, where the frequencies stay near one.  Every angle is
    # good to 1e-6 (times 1 / theta below theta 1); the sine, the cosine and the
    # fp32 products add a few 2^-24 (4e-7) of the pair's magnitudes.
    g = torch.Generator(device="cuda").manual_seed(22)
    n, pairs = 1000, sum(sections)
    q = torch.randn(1, 1, n, 256, generator=g, device="cuda")
    pos = torch.randint((1 << 31) - 100000, 1 << 31, (len(sections), 1, n), generator=g, device="cuda")
    pos[:, :, ::3] *= -1
    got, _ = mgq.rotary(q, None, pos, sections=sections, theta=theta, per_axis=per_axis)
    angle = exact_turns(sections, theta, per_axis, pos[:, 0].tolist()) * (2 * math.pi)
    x, z = (q[0, 0, :, i:i + pairs].double() for i in (0, pairs))
    want = torch.cat([x * angle.cos() - z * angle.sin(), z * angle.cos() + x * angle.sin()], -1)
    mag = (x.abs() + z.abs()).repeat(1, 2)
    lim = (1e-6 * max(1.0, 1.0 / theta) + 4e-7) * mag + 2.0 ** -24 * want.abs()
    over = (got[0, 0, :, :2 * pairs].double() - want).abs() / lim
    assert over.max().item() <= 1.0, over.max().item()


def test_rotary_sections_that_no_int_holds():
    q = torch.zeros(1, 2, 3, 128, device="cuda")
    pos = torch.zeros(1, 1, 3, dtype=torch.int32, device="cuda")
    for sections in ((2 ** 32 + 32,), (2 ** 33,), (-2 ** 32 + 32,), (32.5,)):
        with pytest.raises(ValueError, match="whole numbers"):
            mgq.rotary(q, None, pos, sections=sections)


# ---------------------------------------------------------------- softcap
def saturated(d, low=5.0, high=9.0, cap=20.0, seed=23, b=1, h=2, lq=300, lk=300):
    """q and k whose every |logit / cap| lies in [low, high]."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)

    u = torch.where(uniform(1, 1, 1, d) < 0.5, -1.0, 1.0)
    mid = math.sqrt(low * high) * cap / math.sqrt(d)      # |q| |k| of every element
    half = math.sqrt(high / low) ** 0.5 * (1 - 2.0 ** -7)  # room for the roundings to bf16
    size = [math.sqrt(mid) * half ** (2 * uniform(b, h, n, 1) - 1) for n in (lq, lk)]
    q = (size[0] * u).bfloat16()
    k = (size[1] * u * torch.where(uniform(b, h, lk, 1) < 0.5, -1.0, 1.0)).bfloat16()
    v, do = (torch.randn(b, h, n, d, generator=g, device="cuda").bfloat16() for n in (lk, lq))
    return q, k, v, do


@pytest.mark.parametrize("path,d", [(0, 64), (0, 128), (1, 128), (0, 256)])
@pytest.mark.parametrize("low,high", [(2.0, 4.0), (5.0, 7.0), (7.0, 9.0), (9.0, 11.0)])
@pytest.mark.parametrize("sizes", [dict(), dict(h=16, lq=700, lk=800)], ids=["two terms", "one term"])
def test_gradients_of_saturated_logits(path, d, low, high, sizes):
    cap = 20.0
    q, k, v, do = saturated(d, low, high, cap, **sizes)
    kw = dict(causal=True, window=None, softcap=cap)
    o, lse = mgq.attention_lse(q, k, v, **kw)
    got = forced(path, lambda: mgq.attention_backward(do, q, k, v, o, lse, **kw))
    f = ref.forward(q, k, v, **kw)
    y = torch.where(f["see"], torch.atanh(f["t"].clamp(-1 + 1e-15, 1 - 1e-15)).abs(), torch.zeros_like(f["t"]))
    assert low - 0.01 <= y[y > 0].min() and y.max() <= high + 0.01
    # 1 - tanh^2 without cancellation, 4 e / (1 + e)^2 with e = e^(-2 |y|).
    z = torch.einsum("bhqd,bhkd->bhqk", f["q"], f["k"]) * f["scale"] / cap
    e = torch.exp(-2 * z.abs())
    chain = 4 * e / (1 + e) ** 2
    dod, od = do.double(), o.double()
    p = torch.exp(f["x"] - lse.double()[..., None])
    dp = dod @ f["v"].transpose(-1, -2)
    delta = (dod * od).sum(-1, keepdim=True)
    mag = dod.abs() @ f["v"].abs().transpose(-1, -2) + (dod * od).abs().sum(-1, keepdim=True)
    ds = p * (dp - delta) * chain * f["scale"]
    # Relative errors.  P: its logit's and lse's, as in the reference's bound.  The
    # factor: e is off by twice the error of |y|, which is that of the product
    # (E32 of its magnitudes) and three roundings, and by the approximate
    # exponential, reciprocal and three products, 2^-20 together.
    ep = ref.logit_error(f) + ref.E32 * (1 + lse.double().abs()[..., None] + cap)
    ec = 2 * (ref.E32 * f["mag"] / cap + z.abs() * 2.0 ** -22) + 2.0 ** -20
    err = (ref.U16 + ep + ec) * ds.abs() + f["scale"] * p * chain * ref.E32 * mag
    g = f["group"]
    for n, x, w, b, m in (
            ("dq", got[0], ds @ f["k"], err @ f["k"].abs(), ds.abs() @ f["k"].abs()),
            ("dk", got[1], ref.fold(ds.transpose(-1, -2) @ f["q"], g),
             ref.fold(err.transpose(-1, -2) @ f["q"].abs(), g),
             ref.fold(ds.abs().transpose(-1, -2) @ f["q"].abs(), g))):
        ref.assert_within(n, x, w, (b + 2.0 ** -16 * m + ref.U16 * w.abs()) * (1 + ref.U16) + 1e-30)


@pytest.mark.parametrize("path,d", [(0, 64), (0, 128), (1, 64), (0, 256)])
@pytest.mark.parametrize("cap", [60.0, 80.0, 150.0, 300.0, 1000.0, 1e4, 1e5])
@pytest.mark.parametrize("high", [0.48, 0.96])
@pytest.mark.parametrize("sizes", [dict(), dict(h=16, lq=700, lk=800)], ids=["small", "large"])
def test_logits_below_large_softcaps(path, d, cap, high, sizes):
    # |logit / cap| up to 1/2 and up to 1, the polynomials' ranges.
    q, k, v, do = saturated(d, 0.25, high, cap, seed=30, **sizes)
    check_forward_and_gradients(None, dict(causal=True, window=None, softcap=cap), dict(q=q, k=k, v=v, do=do),
                                path)


@pytest.mark.parametrize("path,d", [(0, 64), (1, 128), (0, 128), (0, 256)])
@pytest.mark.parametrize("cap", [1e-5, 1e-39, 3e38])
@pytest.mark.parametrize("sizes", [(1, 200, 300, 4, 2), (4, 700, 700, 16, 16), (2, 1, 300, 4, 2)], ids=str)
def test_softcaps_at_the_ends_of_their_range(path, d, cap, sizes):
    b, lq, lk, hq, hkv = sizes
    t, kw = make((b, lq, lk, hq, hkv, d, True, None, cap, 1), seed=24)
    t["q"][:, ::2] = 0  # logits of exactly zero
    f = ref.forward(t["q"], t["k"], t["v"], **{**kw, "softcap": cap if cap < 1 else None})
    o, lse = forced(path, lambda: mgq.attention_lse(t["q"], t["k"], t["v"], **kw))
    plain = {**f, "softcap": 0.0 if cap > 1 else cap}
    ref.assert_within("o", o, f["o"], ref.o_bound(plain))
    ref.assert_within("lse", lse, f["lse"], ref.lse_bound(plain))
    got = forced(path, lambda: mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse, **kw))
    want, bound = ref.backward(t["q"], t["k"], t["v"], o, lse, t["do"], None, True, None,
                               cap if cap < 1 else None)
    bound = list(bound)
    if cap < 1:
        # The slope sech^2(y), y = x / cap, also moves with the error of the fp32
        # product x (E32 of its magnitudes): between sech^2(|y| + dy) and
        # sech^2(|y| - dy), which for these caps is all of it near x = 0.
        z = torch.einsum("bhqd,bhkd->bhqk", f["q"], f["k"]).abs() * f["scale"]
        dz = ref.E32 * f["mag"]

        def slope(x):
            e = torch.exp(-2 * (x / cap).clamp(max=300))
            return 4 * e / (1 + e) ** 2

        do, od = t["do"].double(), o.double()
        p = torch.exp(f["x"] - lse.double()[..., None])
        dp = do @ f["v"].transpose(-1, -2) - (do * od).sum(-1, keepdim=True)
        room = p * dp.abs() * (slope((z - dz).clamp(min=0)) - slope(z + dz)) * f["scale"] * (1 + 2 * ref.U16)
        bound[0] = bound[0] + room @ f["k"].abs()
        bound[1] = bound[1] + ref.fold(room.transpose(-1, -2) @ f["q"].abs(), f["group"])
    for n, x, w, r in zip(("dq", "dk", "dv"), got, want, bound):
        ref.assert_within(n, x, w, r)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [1e6, 1e7, 1e8])
@pytest.mark.parametrize("sizes", [(1, 200, 300, 4, 2), (4, 700, 700, 16, 16)], ids=str)
def test_running_maximum_of_huge_logits(d, cap, sizes):
    # Logits of about a third of such caps: a maximum that is off by the hardware
    # tanh's error, times the cap, is off by more than fp32's exponents span.
    t, kw = make((*sizes, d, True, None, cap, 1), seed=25)
    t["q"] = (t["q"].float() * 0.3 * cap).bfloat16()
    f = ref.forward(t["q"], t["k"], t["v"], **kw)
    o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
    assert torch.isfinite(o).all()
    ref.assert_within("lse", lse, f["lse"], ref.lse_bound(f))


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


@pytest.mark.parametrize("case", [c for c in NAN_ROWS if c[8]], ids=str)
def test_a_row_of_minus_infinities_below_the_cap(case):
    # Every visible logit is -inf, which the cap makes -cap: the plain mean of v.
    case, path = dims(case)
    t, kw = make(case, seed=27)
    row = case[1] // 2
    t["k"][..., 3] = -t["k"][..., 3].abs() - 0.01
    t["q"][0, 0, row, 3] = math.inf
    o, lse = forced(path, lambda: mgq.attention_lse(t["q"], t["k"], t["v"], **kw))
    see = ref.visible(case[1], case[2], case[6], case[7], "cuda")[row]
    want = math.log(see.sum().item()) - kw["softcap"]
    assert abs(lse[0, 0, row].item() - want) <= kw["softcap"] * 4e-7 + ref.E32 * (1 + abs(want) + kw["softcap"])
    v = t["v"][0, 0].double()[see]
    assert ((o[0, 0, row].double() - v.mean(0)).abs() <= 2 * ref.U16 * v.abs().mean(0) + 1e-30).all()


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("case", [c for c in NAN_ROWS if c[6]], ids=str)
def test_keys_that_are_not_numbers_leave_the_rows_before_them_alone(case, value):
    case, path = dims(case)
    t, kw = make(case, seed=34)
    f = ref.forward(t["q"], t["k"], t["v"], **kw)
    row = case[1] // 2                             # the first row that sees such a key
    t["k"][:, :, case[2] - case[1] + row:, 1::5] = float(value)
    o, lse = forced(path, lambda: mgq.attention_lse(t["q"], t["k"], t["v"], **kw))
    ref.assert_within("o", o[:, :, :row], f["o"][:, :, :row], ref.o_bound(f)[:, :, :row])
    ref.assert_within("lse", lse[:, :, :row], f["lse"][:, :, :row], ref.lse_bound(f)[:, :, :row])
    if value == "nan" and kw["window"] is None:  # every later row sees one
        assert torch.isnan(lse[:, :, row:]).all()


@pytest.mark.parametrize("path,d,lq", [(0, 64, 256), (0, 128, 256), (0, 128, 200), (1, 128, 256), (0, 256, 256)])
@pytest.mark.parametrize("cap", [None, 50.0])
def test_an_infinite_gradient_reaches_every_visible_key(path, d, lq, cap):
    # Where P has underflowed to zero too (0 * inf), in tiles with a mask as in others.
    lk = lq
    t, kw = make((1, lq, lk, 4, 2, d, True, None, cap, 60), seed=28)
    o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
    row = lq - 40
    t["do"][0, 0, row, 5] = math.inf
    dq, dk, dv = forced(path, lambda: mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse, **kw))
    assert not torch.isfinite(dq[0, 0, row]).any()
    assert torch.isfinite(dq[0, 0, :row]).all() and torch.isfinite(dq[0, 1:]).all()
    assert not torch.isfinite(dk[0, 0, :row + 1]).any()
    assert torch.isfinite(dk[0, 0, row + 1:]).all() and torch.isfinite(dk[0, 1]).all()


# ---------------------------------------------------------------- the chain of kernels
@pytest.mark.parametrize("case", [(1, 128, 128, 4, 1, 128, True, None, None, 1),
                                  (2, 700, 900, 8, 2, 64, True, None, None, 1),
                                  (1, 300, 450, 4, 2, 256, True, 200, None, 1)], ids=str)
def test_every_replay_reads_its_own_statistics(case):
    # The dQ kernel does not wait for the statistics itself: one scratch, inputs in turn.
    sets = []
    for seed in (32, 33):
        t, kw = make(case, seed=seed)
        o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
        args = [t["do"], t["q"], t["k"], t["v"], o, lse]
        sets.append((args, mgq.attention_backward(*args, **kw)))
    now = [torch.empty_like(x) for x in sets[0][0]]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = mgq.attention_backward(*now, **kw)
    for turn in range(100):
        args, want = sets[turn & 1]
        for a, b in zip(now, args):
            a.copy_(b)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), turn


# ---------------------------------------------------------------- arguments
def test_windows_past_32_bits():
    # A window longer than the keys hides none of them; it still is a window.
    t, _ = make((1, 100, 100, 4, 2, 64, False, None, None, 1), seed=29)
    q, k, v = t["q"], t["k"], t["v"]
    o, lse = mgq.attention_lse(q, k, v, causal=True)
    want = mgq.attention_backward(t["do"], q, k, v, o, lse, causal=True)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 7, 2 ** 40):
        r = mgq.attention_lse(q, k, v, window=window)
        assert torch.equal(r[0], o) and torch.equal(r[1], lse)
        got = mgq.attention_backward(t["do"], q, k, v, o, lse, window=window)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(mgq.attention(q, k, v, window=window), mgq.attention(q, k, v, causal=True))


def test_inputs_that_require_a_gradient_are_not_passed_over_in_silence():
    t, _ = make((1, 20, 20, 2, 1, 64, False, None, None, 1), seed=31)
    q, k, v, do = (t[n] for n in ("q", "k", "v", "do"))
    o, lse = mgq.attention_lse(q, k, v)
    pos = torch.zeros(1, 1, 20, dtype=torch.int32, device="cuda")
    kr = k.expand(1, 2, 20, 64).contiguous()
    calls = {"attention_lse": lambda: mgq.attention_lse(q, k, v),
             "attention_backward": lambda: mgq.attention_backward(do, q, k, v, o, lse),
             "rotary": lambda: mgq.rotary(q, kr, pos, sections=(32,))}
    for name, call in calls.items():
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            want = call()
            k.requires_grad_(), kr.requires_grad_()
            with torch.no_grad():
                call()
        with pytest.warns(UserWarning, match=f"^{name} records no autograd graph"):
            got = call()
        k.requires_grad_(False), kr.requires_grad_(False)
        assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, want))
