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
    (1, 417, 417, 6, 2, 64, True, 100, 20.0, 3),       # ragged heads, an odd group
    (2, 1153, 1400, 16, 4, 128, True, None, None, 1),  # ragged heads, more tile pairs than SMs
    # Few tiles, long walks: cut into parts that are joined.
    (1, 3000, 64, 3, 1, 32, False, None, None, 4),     # few keys under many rows
    (2, 1500, 200, 2, 1, 128, True, None, 30.0, 2),    # the same, most rows empty
    (1, 2, 5000, 8, 2, 128, True, None, None, 1),      # few rows over many keys
    (1, 3, 7000, 4, 1, 72, True, 3000, 50.0, 4),       # the same, parts without a visible key
    (1, 1100, 1300, 1, 1, 104, True, None, None, 1),   # both, of uneven length
    (1, 1400, 90, 2, 1, 200, True, None, None, 1),     # wide heads
    (1, 5, 2100, 2, 1, 256, False, 1500, 20.0, 1),
    (1, 700, 16, 16, 4, 256, True, 26, None, 4),       # most rows of wide heads empty
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


def steps(case):
    """Key tiles times row tiles, heads apart (at least what the library counts)."""
    b, lq, lk, hq, _, d = case[:6]
    tile = 64 if d > 128 else 128
    return b * hq * (-(-lq // tile)) * (-(-lk // tile))


@pytest.mark.parametrize("case", [c for c in CASES if steps(c) <= 148], ids=str)
def test_small_problems_keep_two_terms(case):
    # At most 148 steps: P and dS in two bf16 terms.
    t, kw = make(case, seed=13)
    o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
    want, bound = ref.backward(t["q"], t["k"], t["v"], o, lse, t["do"], None, inner=2.0 ** -16, **kw)
    got = mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse, **kw)
    for n, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        ref.assert_within(n, g, w, b)


def test_results_are_deterministic():
    t, kw = make((2, 700, 900, 8, 2, 128, True, 400, 30.0, 3), seed=2, dlse=True)
    o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
    first = mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse, dlse=t["dlse"], **kw)
    for _ in range(5):
        o2, lse2 = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
        again = mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse, dlse=t["dlse"], **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_results_over_disjoint_keys_merge():
    # Two halves of the keys, merged by their statistics, are the whole.
    t, kw = make((2, 65, 700, 8, 2, 128, False, None, None, 2), seed=3)
    q, k, v = t["q"], t["k"], t["v"]
    f = ref.forward(q, k, v, **kw)
    parts = [mgq.attention_lse(q, k[:, :, a:b].contiguous(), v[:, :, a:b].contiguous(), **kw)
             for a, b in ((0, 300), (300, 700))]
    stat = torch.stack([p[1] for p in parts]).double()
    lse = torch.logsumexp(stat, 0)
    o = sum(torch.exp(s - lse)[..., None] * p[0].double() for p, s in zip(parts, stat))
    # Each part's o is rounded once more than the whole's.
    ref.assert_within("o", o, f["o"], 2 * ref.o_bound(f))
    ref.assert_within("lse", lse, f["lse"], 2 * ref.lse_bound(f))


@pytest.mark.parametrize("case", [(1, 150, 200, 4, 2, 128, True, None, None, 2),
                                  (1, 90, 130, 2, 1, 64, True, 50, 20.0, 4)], ids=str)
def test_gradients_against_differences(case):
    # Central differences of the fp64 forward pass along random directions.
    t, kw = make(case, seed=4)
    q, k, v, do = t["q"], t["k"], t["v"], t["do"]
    o, lse = mgq.attention_lse(q, k, v, **kw)
    got = mgq.attention_backward(do, q, k, v, o, lse, **kw)
    _, bound = ref.backward(q, k, v, o, lse, do, None, **kw)
    # delta takes the rounded o, the true gradient the exact one.
    f = ref.forward(q, k, v, **kw)
    off = (do.double().abs() * (f["o"] - o.double()).abs()).sum(-1, keepdim=True)
    ds = f["p"] * off * f["scale"]
    extra = (ds @ f["k"].abs(), ref.fold(ds.transpose(-1, -2) @ f["q"].abs(), f["group"]),
             torch.zeros_like(v, dtype=torch.float64))
    g = torch.Generator(device="cuda").manual_seed(5)
    for i, x in enumerate((q, k, v)):
        u = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4

        def loss(step):
            args = [a.double() for a in (q, k, v)]
            args[i] = args[i] + step * u
            return (ref.forward(*args, **kw)["o"] * do.double()).sum().item()

        slope = (loss(h) - loss(-h)) / (2 * h)
        mine = (got[i].double() * u).sum().item()
        room = ((bound[i] + extra[i]) * u.abs()).sum().item()
        assert abs(mine - slope) <= room + 1e-5 * abs(slope), (i, mine, slope, room)


def test_empty_sizes():
    def z(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")

    for b, lq, lk in ((0, 4, 4), (2, 0, 5), (2, 5, 0)):
        q, k = z(b, 4, lq, 64), z(b, 2, lk, 64)
        o, lse = mgq.attention_lse(q, k, k.clone(), causal=True)
        assert o.shape == q.shape and (o == 0).all()
        assert (lse == -float("inf")).all()
        dq, dk, dv = mgq.attention_backward(z(*q.shape), q, k, k.clone(), o, lse, causal=True,
                                            dk=torch.ones_like(k), dv=torch.ones_like(k))
        assert (dq == 0).all() and (dk == 0).all() and (dv == 0).all()


def test_outputs_given_and_their_surroundings():
    t, kw = make((1, 77, 130, 4, 2, 72, True, 60, None, 1), seed=6)
    q, k, v = t["q"], t["k"], t["v"]
    want_o, want_lse = mgq.attention_lse(q, k, v, **kw)
    want = mgq.attention_backward(t["do"], q, k, v, want_o, want_lse, **kw)

    def inside(x):
        pad = 4096
        buf = torch.full((x.numel() + 2 * pad,), 7.0, dtype=x.dtype, device="cuda")
        return buf, buf[pad:pad + x.numel()].view(x.shape), pad

    made = [inside(x) for x in (want_o, want_lse, *want)]
    o, lse, dq, dk, dv = (m[1] for m in made)
    r = mgq.attention_lse(q, k, v, out=o, lse=lse, **kw)
    assert r[0] is o and r[1] is lse
    r = mgq.attention_backward(t["do"], q, k, v, o, lse, dq=dq, dk=dk, dv=dv, **kw)
    assert r[0] is dq and r[1] is dk and r[2] is dv
    for (buf, x, pad), w in zip(made, (want_o, want_lse, *want)):
        assert torch.equal(x, w)
        assert (buf[:pad] == 7).all() and (buf[pad + x.numel():] == 7).all()


def test_two_streams_at_once():
    cases = [(2, 500, 700, 8, 2, 128, True, None, None, 1), (1, 1200, 1200, 4, 4, 64, False, None, None, 1)]
    sets, streams = [make(c, seed=7 + i) for i, c in enumerate(cases)], [torch.cuda.Stream() for _ in cases]
    want = []
    for t, kw in sets:
        o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
        want.append((o, lse, *mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse, **kw)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):  # the stream as an argument; nothing waits in between
        for i, (t, kw) in enumerate(sets):
            o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], stream=streams[i], **kw)
            got[i].append((o, lse, *mgq.attention_backward(
                t["do"], t["q"], t["k"], t["v"], o, lse, stream=streams[i], **kw)))
    torch.cuda.synchronize()
    for w, rounds in zip(want, got):
        for r in rounds:
            assert all(torch.equal(a, b) for a, b in zip(w, r))


@pytest.mark.parametrize("d", [128, 256])
def test_captured_backward_replays_without_a_direct_call(d):
    t, kw = make((1, 300, 450, 4, 2, d, True, 200, None, 1), seed=8)
    q, k, v, do = t["q"], t["k"], t["v"], t["do"]
    o, lse = mgq.attention_lse(q, k, v, **kw)
    torch.cuda.synchronize()
    # Two graphs captured on one stream, each with its own scratch, replayed on two.
    s = torch.cuda.Stream()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(mgq.attention_backward(do, q, k, v, o, lse, **kw))
        graphs.append(g)
    for seed in (9, 10):
        n, _ = make((1, 300, 450, 4, 2, d, True, 200, None, 1), seed=seed)
        for name, x in (("q", q), ("k", k), ("v", v), ("do", do)):
            x.copy_(n[name])
        o2, lse2 = mgq.attention_lse(q, k, v, **kw)
        o.copy_(o2)
        lse.copy_(lse2)
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(5):
            with torch.cuda.stream(a):
                graphs[0].replay()
            with torch.cuda.stream(b):
                graphs[1].replay()
        torch.cuda.synchronize()
        want = mgq.attention_backward(do, q, k, v, o, lse, **kw)
        for r in outs:
            assert all(torch.equal(x, y) for x, y in zip(r, want))
    assert mgq.status() & 0x1f == 0


def test_what_follows_on_the_stream_finds_every_gradient():
    # The dQ kernel may start, and end its work, before the dK/dV kernel ends:
    # many keys and few rows make dQ the short one.
    t, kw = make((1, 16, 60000, 8, 8, 128, False, None, None, 1), seed=11)
    o, lse = mgq.attention_lse(t["q"], t["k"], t["v"], **kw)
    want = None
    for _ in range(10):
        grads = [torch.full_like(t[n], float("nan")) for n in ("q", "k", "v")]
        mgq.attention_backward(t["do"], t["q"], t["k"], t["v"], o, lse, dq=grads[0], dk=grads[1],
                               dv=grads[2], **kw)
        copies = [g.clone() for g in grads]
        want = want or copies
        assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(copies, want))


def test_offsets_past_32_bits():
    # 2.2e9 elements in k, v and their gradients: the last unit against the reference.
    b, hkv, lk, d = 33, 8, 65600, 128
    assert b * hkv * lk * d > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(12)
    q = torch.randn(b, hkv, 2, d, generator=g, device="cuda").bfloat16()
    do = torch.randn(b, hkv, 2, d, generator=g, device="cuda").bfloat16()
    k, v = (torch.empty(b, hkv, lk, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
            for _ in range(2))
    o, lse = mgq.attention_lse(q, k, v)
    got = mgq.attention_backward(do, q, k, v, o, lse)
    sl = (slice(b - 1, b), slice(hkv - 1, hkv))
    part = [x[sl].contiguous() for x in (q, k, v, o, lse, do)]
    f = ref.forward(*part[:3], False, None, None)
    ref.assert_within("lse", part[4], f["lse"], ref.lse_bound(f))
    want, bound = ref.backward(*part, None, False, None, None)
    for n, x, w, r in zip(("dq", "dk", "dv"), got, want, bound):
        ref.assert_within(n, x[sl], w, r)
