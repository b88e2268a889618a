"""64-bit references of the training operators and how far a kernel may be off.

A rounding to bf16 is off by at most half a step, 2^-8 relative; the kernels
round P and dS to bf16 for the tensor cores (on small problems to two bf16
terms, 2^-16 together) and every output once.  What is
held in fp32 (products summed over head_dim, exponentials, the row
statistics) is given 2^-18 of the sum of the magnitudes involved: 2^-24 a
rounding, for the up to 256 / 16 + 16 partial sums and the approximate
exponential's 2^-22.  The bounds below add these up term by term.
"""
import math

import torch

U16 = 2.0 ** -8
E32 = 2.0 ** -18


def visible(lq, lk, causal, window, device):
    pos = torch.arange(lq, device=device)[:, None] + (lk - lq)
    key = torch.arange(lk, device=device)[None, :]
    see = torch.ones(lq, lk, dtype=torch.bool, device=device)
    if causal or window:
        see &= key <= pos
    if window:
        see &= pos - key < window
    return see


def forward(q, k, v, causal, window, softcap):
    """fp64 (o, lse) and what the bounds need."""
    q, k, v = q.double(), k.double(), v.double()
    b, hq, lq, d = q.shape
    group = hq // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    scale = 1.0 / math.sqrt(d)
    x = torch.einsum("bhqd,bhkd->bhqk", q, k) * scale
    mag = torch.einsum("bhqd,bhkd->bhqk", q.abs(), k.abs()) * scale  # rounding scale of x
    t = torch.zeros_like(x)
    if softcap:
        t = torch.tanh(x / softcap)
        x = softcap * t
    see = visible(lq, k.shape[2], causal, window, q.device)
    x = x.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(x, -1) if k.shape[2] else torch.full(q.shape[:3], -math.inf).to(q)
    base = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
    p = torch.exp(x - base[..., None])
    return dict(q=q, k=k, v=v, x=x, t=t, mag=mag, see=see, lse=lse, p=p, o=p @ v, scale=scale,
                group=group, softcap=softcap or 0.0)


def logit_error(f):
    """Error of a logit: its product's, the softcap's tanh (4e-7 absolute, times the cap)."""
    return E32 * (1.0 + f["mag"]) + f["softcap"] * 4e-7


def lse_bound(f):
    """A row's log-sum-exp is off by at most its largest logit error, and its own rounding."""
    err = torch.where(f["see"], logit_error(f), torch.zeros_like(f["x"])).amax(-1)
    lse = f["lse"].abs()
    return err + E32 * (1.0 + torch.where(torch.isinf(lse), torch.zeros_like(lse), lse))


def o_bound(f):
    return (U16 + E32 + 2 * (f["p"] * logit_error(f)).amax(-1, keepdim=True)) * (f["p"] @ f["v"].abs()) \
        + U16 * f["o"].abs() + 1e-30


def fold(x, group):
    """Sums over the q heads of each kv head."""
    b, h = x.shape[:2]
    return x.view(b, h // group, group, *x.shape[2:]).sum(2)


def backward(q, k, v, o, lse, do, dlse, causal, window, softcap, inner=U16):
    """fp64 gradients from the statistics given, and their bounds; ``inner`` is
    the relative rounding of P and dS."""
    f = forward(q, k, v, causal, window, softcap)
    do, o = do.double(), o.double()
    stat = lse.double()
    dead = stat == -math.inf
    p = torch.exp(f["x"] - torch.where(dead, torch.zeros_like(stat), stat)[..., None])
    p = torch.where(dead[..., None], torch.zeros_like(p), p)
    dp = do @ f["v"].transpose(-1, -2)
    dp_mag = do.abs() @ f["v"].abs().transpose(-1, -2) + (do * o).abs().sum(-1, keepdim=True)
    delta = (do * o).sum(-1, keepdim=True)
    if dlse is not None:
        delta = delta - dlse.double()[..., None]
        dp_mag = dp_mag + dlse.double().abs()[..., None]
    chain = 1.0 - f["t"] ** 2
    ds = p * (dp - delta) * chain * f["scale"]
    # Relative error of p: its logit's and lse's rounding in log2 units.
    finite = torch.where(torch.isinf(stat), torch.zeros_like(stat), stat).abs()[..., None]
    xmag = torch.where(f["see"], f["x"], torch.zeros_like(f["x"])).abs()
    ep = logit_error(f) + E32 * (1.0 + finite + xmag)
    p_err = (inner + ep) * p
    ds_err = (inner + ep) * ds.abs() + f["scale"] * p * E32 * dp_mag * chain \
        + f["scale"] * p * (dp - delta).abs() * 1e-6
    g = f["group"]
    dq = ds @ f["k"]
    dk = fold(ds.transpose(-1, -2) @ f["q"], g)
    dv = fold(p.transpose(-1, -2) @ do, g)
    sum32 = 2.0 ** -16  # fp32 sums over up to some thousands of rows or keys
    dq_mag = ds.abs() @ f["k"].abs()
    dk_mag = fold(ds.abs().transpose(-1, -2) @ f["q"].abs(), g)
    dv_mag = fold(p.transpose(-1, -2) @ do.abs(), g)
    bq = ds_err @ f["k"].abs() + sum32 * dq_mag + U16 * dq.abs() + 1e-30
    bk = fold(ds_err.transpose(-1, -2) @ f["q"].abs(), g) + sum32 * dk_mag + U16 * dk.abs() + 1e-30
    bv = fold(p_err.transpose(-1, -2) @ do.abs(), g) + sum32 * dv_mag + U16 * dv.abs() + 1e-30
    # The output's rounding applies to the value with its error.
    return (dq, dk, dv), tuple(b * (1 + U16) for b in (bq, bk, bv))


def assert_within(name, got, want, bound):
    got = got.double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - want).abs() / bound
    worst = over.max().item() if over.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound at {int(over.argmax())}"
