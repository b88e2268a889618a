"""The operators as they are used together (GPU): a training step's chain
rotary -> attention -> backward -> inverse rotary, and a decode step whose new
token is turned before it enters the cache."""
import pytest
import torch

import masked_grouped_query_b200 as mgq
from tests import training_reference as ref
from tests.test_rotary_gpu import reference

pytestmark = pytest.mark.gpu

ROT = dict(sections=(12, 10, 10), theta=10000.0, per_axis=False, interleaved=False)


def turned(x, pos, inverse=False):
    """fp64 rotation of (batch, length, heads, d), differentiable."""
    return reference(x, pos, seq_major=True, inverse=inverse, **ROT)[0]


def inputs(b=2, length=300, hq=4, hkv=2, d=64):
    g = torch.Generator(device="cuda").manual_seed(5)

    def randn(h):
        return (torch.randn(b, length, h, d, generator=g, device="cuda")).bfloat16()

    t = torch.arange(length, device="cuda")
    pos = torch.stack([t // 60, (t // 10) % 6, t % 10])[:, None].repeat(1, b, 1).int().contiguous()
    return randn(hq), randn(hkv), randn(hkv), randn(hq).transpose(1, 2).contiguous(), pos


@pytest.mark.parametrize("captured", [False, True])
def test_training_step(captured):
    q, k, v, do, pos = inputs()
    kw = dict(causal=True, window=120)

    def step():
        qr, kr = mgq.rotary(q, k, pos, seq_major=True, out_seq_major=False, **ROT)
        vr = v.transpose(1, 2).contiguous()
        o, lse = mgq.attention_lse(qr, kr, vr, **kw)
        dq, dk, dv = mgq.attention_backward(do, qr, kr, vr, o, lse, **kw)
        gq, gk = mgq.rotary(dq, dk, pos, inverse=True, seq_major=False, out_seq_major=True, **ROT)
        return o, gq, gk, dv.transpose(1, 2).contiguous()

    if captured:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step()  # sizes the stream's split workspace
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
        graph.replay()
    else:
        got = step()
    torch.cuda.synchronize()
    # fp64, through autograd, with the rounding that the chain makes at the
    # rotary's output.
    leaves = [x.double().requires_grad_() for x in (q, k, v)]
    f = ref.forward(turned(leaves[0], pos).transpose(1, 2), turned(leaves[1], pos).transpose(1, 2),
                    leaves[2].transpose(1, 2), True, 120, None)
    (f["o"] * do.double()).sum().backward()
    want = (f["o"].detach(), *[x.grad for x in leaves])
    # Along the chain: the turned q and k are rounded (half a step, 2^-8, each),
    # which moves a logit by 2 * 2^-8 of its products' root sum of squares, below
    # 0.02 for these inputs, and P with it; then P or dS, o, the gradient and
    # its turned value are rounded.  0.02 + 4 * 2^-8 in the 2-norm.
    for n, a, w in zip(("o", "dq", "dk", "dv"), got, want):
        rel = ((a.double() - w).norm() / w.norm()).item()
        assert rel <= 0.02 + 4 * 2.0 ** -8, (n, rel)


def test_decode_step_on_a_cache():
    # A projection's fp32 token is turned, appended and attended to.
    b, slots, hq, hkv, d, at = 3, 128, 8, 2, 64, 100
    g = torch.Generator(device="cuda").manual_seed(6)
    kc, vc = (torch.randn(b, slots, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q, k, v = (torch.randn(b, 1, h, d, generator=g, device="cuda") for h in (hq, hkv, hkv))
    pos = torch.full((1, b, 1), at, dtype=torch.int32, device="cuda")
    qb, _ = mgq.rotary(q, None, pos, sections=(32,), seq_major=True, out_seq_major=False,
                       out_dtype=torch.bfloat16)
    _, kr = mgq.rotary(q, k, pos, sections=(32,), seq_major=True)
    k2, v2 = kc.clone(), vc.clone()
    o = mgq.decode_append(qb, k2, v2, kr, v, at)
    rot = dict(sections=(32,), theta=10000.0, per_axis=False, interleaved=False, inverse=False)
    want_k = reference(k, pos, seq_major=True, **rot)[0]
    assert ((k2[:, at].double() - want_k[:, 0]).abs() <= 2.0 ** -8 * want_k[:, 0].abs() + 1e-5).all()
    f = ref.forward(qb, k2[:, :at + 1].transpose(1, 2), v2[:, :at + 1].transpose(1, 2), True, None, None)
    ref.assert_within("o", o, f["o"], ref.o_bound(f))
