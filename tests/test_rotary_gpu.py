"""rotary against a 64-bit reference (GPU)."""
import pytest
import torch

import masked_grouped_query_b200 as mgq

pytestmark = pytest.mark.gpu

# An angle is off by at most 1e-6 (positions of 32 bits), its sine and cosine
# and the two fp32 products by a few 2^-24: 1.4e-6 of the pair's magnitudes;
# then one rounding to the output's type.
ANGLE = 1.4e-6


def reference(x, positions, sections, theta, per_axis, interleaved, inverse, seq_major):
    """fp64 (batch, length, heads, d) and the magnitude of every element's pair."""
    x = x.double() if seq_major else x.double().transpose(1, 2)
    pairs = sum(sections)
    freq, axis = [], []
    for a, s in enumerate(sections):
        for j in range(s):
            freq.append(theta ** (-(j / s) if per_axis else -(len(freq) / pairs)))
            axis.append(a)
    angle = positions.double()[axis].permute(1, 2, 0) * torch.tensor(freq, dtype=torch.float64,
                                                                     device=x.device)
    c, s = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
    if inverse:
        s = -s
    i0, i1 = ((slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved
              else (slice(0, pairs), slice(pairs, 2 * pairs)))
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    mag[..., i0] = mag[..., i1] = x[..., i0].abs() + x[..., i1].abs()
    return y, mag


def check(got, x, positions, seq_major, out_seq_major, **kw):
    want, mag = reference(x, positions, seq_major=seq_major, **kw)
    got = got if out_seq_major else got.transpose(1, 2)
    half = torch.finfo(got.dtype).eps / 2
    over = (got.double() - want).abs() / (ANGLE * mag + half * want.abs() * (1 + ANGLE)
                                          + half * ANGLE * mag + 1e-38)
    assert torch.isfinite(got).all() and over.max().item() <= 1.0, over.max().item()


CASES = [
    # (batch, length, hq, hkv, d, sections, seq_major, out_seq_major, interleaved, per_axis)
    (1, 1, 1, 0, 8, (4,), False, False, False, False),
    (3, 1, 8, 2, 128, (16, 24, 24), True, False, False, False),
    (2, 5, 4, 1, 128, (64,), True, True, True, False),
    (1, 37, 6, 2, 72, (18, 18), False, False, False, True),
    (2, 130, 3, 3, 72, (5, 6, 7), False, True, True, True),      # odd sections, tail passed through
    (1, 9, 2, 1, 256, (32,), True, False, False, False),         # a quarter of the head turns
    (1, 700, 16, 16, 80, (8, 16, 8, 8), False, False, False, False),
    (5, 3, 1, 1, 16, (1, 1), False, True, True, False),
    (1, 2000, 32, 8, 128, (16, 24, 24), True, False, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtypes", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                    (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)],
                         ids=["bf16", "fp32", "fp32-bf16", "bf16-fp32"])
def test_rotary(case, dtypes):
    b, length, hq, hkv, d, sections, sm, osm, inter, per_axis = case
    g = torch.Generator(device="cuda").manual_seed(length)
    shape = (lambda h: (b, length, h, d)) if sm else (lambda h: (b, h, length, d))
    q = torch.randn(shape(hq), generator=g, device="cuda").to(dtypes[0])
    k = torch.randn(shape(hkv), generator=g, device="cuda").to(dtypes[0]) if hkv else None
    for far, itype in ((1 << 31, torch.int64), (5000, torch.int32)):
        pos = torch.randint(-far + 1, far, (len(sections), b, length), generator=g,
                            device="cuda").to(itype)
        for inverse in (False, True):
            kw = dict(sections=sections, theta=10000.0, per_axis=per_axis, interleaved=inter,
                      inverse=inverse)
            qo, ko = mgq.rotary(q, k, pos, seq_major=sm, out_seq_major=osm, out_dtype=dtypes[1], **kw)
            assert qo.dtype == dtypes[1]
            check(qo, q, pos, sm, osm, **kw)
            if hkv:
                check(ko, k, pos, sm, osm, **kw)
            else:
                assert ko is None


def test_in_place_and_back_again():
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, 4, 50, 128, generator=g, device="cuda")
    k = torch.randn(2, 2, 50, 128, generator=g, device="cuda")
    pos = torch.randint(0, 1 << 20, (3, 2, 50), generator=g, device="cuda")
    want = mgq.rotary(q, k, pos, sections=(16, 24, 20))
    a, b = q.clone(), k.clone()
    r = mgq.rotary(a, b, pos, sections=(16, 24, 20), out=(a, b))
    assert r[0] is a and r[1] is b
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert torch.equal(a[..., 120:], q[..., 120:])      # the tail stays
    back = mgq.rotary(a, b, pos, sections=(16, 24, 20), inverse=True)
    # Two rotations, each off by at most ANGLE and a rounding of the pair's magnitudes.
    for x, y in zip(back, (q, k)):
        lim = 4 * (ANGLE + 2.0 ** -24) * (x.abs() + y.abs() + y.abs().max())
        assert ((x - y).abs() <= lim).all()


def test_positions_of_the_smallest_and_largest_calls():
    # No tokens; and more than 2^31 elements, the last rows against the reference.
    q = torch.zeros(0, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    qo, _ = mgq.rotary(q, None, torch.zeros(1, 0, 3, dtype=torch.int32, device="cuda"), sections=(32,))
    assert qo.shape == q.shape
    length, heads = 70400, 240
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.empty(1, length, heads, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert q.numel() > 1 << 31
    pos = torch.randint(0, 1 << 30, (2, 1, length), generator=g, device="cuda").int()
    kw = dict(sections=(30, 34), theta=1e6, per_axis=False, interleaved=False, inverse=False)
    qo, _ = mgq.rotary(q, None, pos, seq_major=True, out_seq_major=False, **kw)
    check(qo[:, :, -5:].contiguous(), q[:, -5:].contiguous(), pos[:, :, -5:].contiguous(), True, False, **kw)


def test_captured_call_and_given_stream():
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(4, 1, 8, 128, generator=g, device="cuda")
    k = torch.randn(4, 1, 2, 128, generator=g, device="cuda")
    pos = torch.randint(0, 1000, (1, 4, 1), generator=g, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = mgq.rotary(q, k, pos, sections=(64,), seq_major=True, out_dtype=torch.bfloat16)
    for _ in range(3):
        pos += 1
        graph.replay()
        torch.cuda.synchronize()
        want = mgq.rotary(q, k, pos, sections=(64,), seq_major=True, out_dtype=torch.bfloat16, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
