"""Training operators of masked grouped-query attention: what is measured.

Three operators that a training step or a server runs around this package's
attention forward, each in a plain form (elementary torch operations in 32
bits, rounded once at the end) and as the calls that a user makes:

* ``lse``: the forward pass that also returns every row's log-sum-exp, the
  statistic that the backward pass and the merge of partial results read;
* ``backward``: the gradients of q, k and v from q, k, v, o, the rows'
  log-sum-exp and the gradient of o, recomputing the probabilities;
* ``rotary``: rotary positions with one or several axes applied to q and k
  (time, height and width of video tokens, rows and columns of image tokens),
  and the inverse rotation, which is its gradient.
"""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


# ---------------------------------------------------------------- cases
def _attn(op, name, batch, q_len, kv_len, hq, hkv, d, causal, window, softcap, spread=1.0):
    case = dict(op=op, batch=batch, q_len=q_len, kv_len=kv_len, hq=hq, hkv=hkv, d=d,
                causal=causal, window=window, softcap=softcap, spread=spread)
    return case if name is None else dict(name=name, **case)


def _rot(name, batch, length, hq, hkv, d, sections, start, seq_major, out_seq_major, interleaved,
         per_axis, inverse, dtype):
    case = dict(op="rotary", batch=batch, length=length, hq=hq, hkv=hkv, d=d,
                sections=sections, start=start, seq_major=seq_major, out_seq_major=out_seq_major,
                interleaved=interleaved, per_axis=per_axis, inverse=inverse, dtype=dtype)
    return case if name is None else dict(name=name, **case)


def listed():
    return [
        # The smallest training step: one 128-token prompt, where launches and latency count.
        _attn("backward", "backward_tiny_causal", 1, 128, 128, 4, 1, 128, True, 0, 0.0),
        # The image encoder's attention: 729 patches, 16 heads of 72, no mask, heads not shared.
        _attn("backward", "backward_siglip_encoder", 32, 729, 729, 16, 16, 72, False, 0, 0.0),
        # The windowed, softcapped prefill trained: 8 q heads share a kv head.
        _attn("backward", "backward_window_softcap", 2, 4096, 4096, 32, 4, 128, True, 1024, 50.0, 3.0),
        # Ordinary causal training on one long sequence, the largest case.
        _attn("backward", "backward_causal_long", 1, 8192, 8192, 32, 8, 128, True, 0, 0.0),
        # Wide heads, ragged lengths, keys from an earlier chunk in front of the queries.
        _attn("backward", "backward_wide_heads_ragged", 2, 1001, 1501, 8, 4, 256, True, 700, 0.0, 2.0),
        # The training forward of the long sequences: o and the statistics for the backward pass.
        _attn("lse", "lse_causal_prefill", 2, 4096, 4096, 32, 8, 128, True, 0, 0.0),
        # Single-token decode whose result is merged with another device's share of the keys.
        _attn("lse", "lse_decode", 16, 1, 8192, 32, 8, 128, True, 0, 0.0),
        # Softcapped windowed prefill with statistics; logits large enough to reach the cap.
        _attn("lse", "lse_window_softcap", 2, 2047, 2047, 32, 4, 128, True, 1024, 30.0, 6.0),
        # One decode step of video tokens: time, height and width positions, fp32 projections.
        _rot("rotary_decode_step", 16, 1, 32, 8, 128, "16,24,24", 100000, True, True, False, False,
             False, "fp32"),
        # The image encoder's queries and keys on a 27 x 27 grid of patches, two axes.
        _rot("rotary_siglip_grid", 32, 729, 16, 16, 72, "18,18", 0, False, False, False, True,
             False, "bf16"),
        # A long video prompt, token-major from the projection, head-major for the attention.
        _rot("rotary_video_prompt", 2, 16384, 32, 8, 128, "16,24,24", 500000, True, False, False,
             False, False, "bf16"),
        # The gradient of a long text prompt's rotary: head-major in, token-major out, pairs interleaved.
        _rot("rotary_gradient_interleaved", 4, 4001, 32, 8, 128, "64", 0, False, True, True, False,
             True, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["backward", "backward", "lse", "rotary"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8, 16])
    if op == "rotary":
        d = rng.choice([64, 72, 80, 96, 128, 256])
        pairs = d // 2 if rng.random() < 0.7 else d // 4
        axes = rng.choice([1, 2, 3])
        a = pairs // axes
        sections = [a] * (axes - 1) + [pairs - a * (axes - 1)]
        batch = rng.choice([1, 2, 5, 16])
        length = min(_log(rng, 1, 16384), max(1, (1 << 27) // (batch * (hq + hkv) * d)))
        return _rot(None, batch, length, hq, hkv, d, ",".join(str(s) for s in sections),
                    _log(rng, 1, 500000), rng.random() < 0.5, rng.random() < 0.5,
                    rng.random() < 0.3, rng.random() < 0.5, rng.random() < 0.4,
                    rng.choice(["bf16", "bf16", "fp32"]))
    d = rng.choice([32, 64, 72, 96, 128, 128, 256])
    batch = rng.choice([1, 1, 2, 3])
    q_len = _log(rng, 1, 8192)
    # Two keys at least: with one, the gradients of q and k are zero but for rounding.
    kv_len = max(2, q_len) if rng.random() < 0.5 else _log(rng, 2, 8192)
    if d > 128:
        q_len, kv_len = min(q_len, 2048), min(kv_len, 2048)
    # As many (row, key) pairs and as large gradients as the largest listed case at most.
    while batch * hq * q_len * kv_len * d > 32 * 4096 * 8192 * 128 or batch * hq * q_len * kv_len > 1 << 31:
        if batch > 1:
            batch = 1
        elif hq > hkv:
            hq = hkv
        elif hkv > 1:
            hq = hkv = hkv // 2
        else:
            q_len, kv_len = q_len // 2, kv_len // 2
    causal = rng.random() < 0.7
    window = _log(rng, 2, 2048) if rng.random() < 0.35 else 0
    softcap = rng.choice([20.0, 30.0, 50.0]) if rng.random() < 0.35 else 0.0
    return _attn(op, None, batch, q_len, kv_len, hq, hkv, d, causal, window, softcap,
                 rng.choice([1.0, 1.0, 2.0, 4.0]))


# ---------------------------------------------------------------- inputs
def _visible(case, device):
    """(q_len, kv_len) truth values: which keys a query sees (bottom-right aligned)."""
    lq, lk = case["q_len"], case["kv_len"]
    pos = torch.arange(lq, device=device)[:, None] + (lk - lq)
    key = torch.arange(lk, device=device)[None, :]
    see = torch.ones(lq, lk, dtype=torch.bool, device=device)
    if case["causal"]:
        see = see & (key <= pos)
    if case["window"] > 0:
        see = see & (key <= pos) & (pos - key < case["window"])
    return see


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(shape, spread=1.0, dtype=BF16):
        return (torch.randn(shape, generator=g, device=dev) * spread).to(dtype)

    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    if case["op"] == "rotary":
        dt = BF16 if case["dtype"] == "bf16" else torch.float32
        length = case["length"]
        sections = [int(s) for s in case["sections"].split(",")]
        qs = (b, length, hq, d) if case["seq_major"] else (b, hq, length, d)
        ks = (b, length, hkv, d) if case["seq_major"] else (b, hkv, length, d)
        # Tokens of a grid (27 columns): the last axes are row and column, the first runs on.
        t = torch.arange(length, device=dev) + case["start"]
        axes = [t] if len(sections) == 1 else [(t // 27) % 27, t % 27]
        if len(sections) == 3:
            axes = [t // 729] + axes
        shift = torch.randint(0, 1000, (1, b, 1), generator=g, device=dev)
        positions = (torch.stack(axes)[:, None, :] + shift).to(torch.int32).contiguous()
        return dict(case=case, q=randn(qs, dtype=dt), k=randn(ks, dtype=dt), positions=positions,
                    sections=sections)
    lq, lk = case["q_len"], case["kv_len"]
    st = dict(case=case, q=randn((b, hq, lq, d), case["spread"]), k=randn((b, hkv, lk, d)),
              v=randn((b, hkv, lk, d)))
    if case["op"] == "backward":
        st["do"] = randn((b, hq, lq, d))
        # What a training step has kept from its forward pass.
        st["o"], st["lse"] = _plain_lse(st)
    return st


# ---------------------------------------------------------------- plain forms
def _logits(st):
    """fp32 logits of (b, kv head, group * q_len rows, kv_len), hidden keys -inf; tanh of the cap."""
    case, q, k = st["case"], st["q"], st["k"]
    b, hq, lq, d = q.shape
    hkv, lk = k.shape[1], k.shape[2]
    x = q.reshape(b, hkv, -1, d).float() @ k.float().transpose(-1, -2)
    x = x * (1.0 / math.sqrt(d))
    t = None
    if case["softcap"] > 0:
        t = torch.tanh(x / case["softcap"])
        x = t * case["softcap"]
    if case["causal"] or case["window"] > 0:
        x = x.view(b, hkv, hq // hkv, lq, lk).masked_fill(~_visible(case, q.device), -math.inf)
        x = x.view(b, hkv, -1, lk)
    return x, t


def _plain_lse(st):
    q, v = st["q"], st["v"]
    x, _ = _logits(st)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    s = e.sum(-1, keepdim=True)
    o = (e @ v.float()) / torch.where(s == 0, torch.ones_like(s), s)
    lse = torch.log(s) + m
    return o.to(BF16).view(q.shape), lse.view(q.shape[:3])


def _plain_backward(st):
    q, k, v, o, do, lse = st["q"], st["k"], st["v"], st["o"], st["do"], st["lse"]
    b, hq, lq, d = q.shape
    hkv, lk = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d)
    x, t = _logits(st)
    rows = lse.reshape(b, hkv, -1, 1)
    p = torch.exp(x - torch.where(rows == -math.inf, torch.zeros_like(rows), rows))
    del x
    dor = do.float().reshape(b, hkv, -1, d)
    dv = p.transpose(-1, -2) @ dor
    ds = dor @ v.float().transpose(-1, -2)
    ds = ds - (dor * o.float().reshape(b, hkv, -1, d)).sum(-1, keepdim=True)
    ds = ds * p
    if t is not None:
        ds = ds * (1 - t * t)
    dq = (ds @ k.float()) * scale
    dk = (ds.transpose(-1, -2) @ q.float().reshape(b, hkv, -1, d)) * scale
    return dq.to(BF16).view(q.shape), dk.to(BF16), dv.to(BF16)


def _frequencies(case, sections, device):
    """Per pair: its axis and its frequency, in 64 bits."""
    pairs = sum(sections)
    axis = torch.cat([torch.full((s,), i, dtype=torch.long) for i, s in enumerate(sections)])
    if case["per_axis"]:
        expo = torch.cat([torch.arange(s, dtype=torch.float64) / s for s in sections])
    else:
        expo = torch.arange(pairs, dtype=torch.float64) / pairs
    return axis.to(device), torch.pow(torch.tensor(10000.0, dtype=torch.float64), -expo).to(device)


def _plain_rotate(x, cos, sin, pairs, case):
    """x (b, l, h, d) or (b, h, l, d) rotated in fp32, in the layout that is asked for."""
    dt = x.dtype
    if case["seq_major"]:
        c, s = cos[:, :, None, :], sin[:, :, None, :]
    else:
        c, s = cos[:, None, :, :], sin[:, None, :, :]
    xf = x.float()
    if case["interleaved"]:
        a, z = xf[..., 0:2 * pairs:2], xf[..., 1:2 * pairs:2]
        r = torch.stack([a * c - z * s, z * c + a * s], -1).flatten(-2)
    else:
        a, z = xf[..., :pairs], xf[..., pairs:2 * pairs]
        r = torch.cat([a * c - z * s, z * c + a * s], -1)
    y = torch.cat([r, xf[..., 2 * pairs:]], -1)
    if case["seq_major"] != case["out_seq_major"]:
        y = y.transpose(1, 2)
    return y.to(dt).contiguous()


def _plain_rotary(st):
    case = st["case"]
    pairs = sum(st["sections"])
    axis, freq = _frequencies(case, st["sections"], st["q"].device)
    # Angles in 64 bits: 32 lose the fraction of a turn at far positions.
    angle = st["positions"].double()[axis].permute(1, 2, 0) * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if case["inverse"]:
        sin = -sin
    return (_plain_rotate(st["q"], cos, sin, pairs, case),
            _plain_rotate(st["k"], cos, sin, pairs, case))


# ---------------------------------------------------------------- the calls
def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "rotary":
            return _plain_rotary(state)
        return _plain_lse(state) if case["op"] == "lse" else _plain_backward(state)
    import masked_grouped_query_b200 as mgq
    if case["op"] == "rotary":
        return mgq.rotary(state["q"], state["k"], state["positions"], sections=state["sections"],
                          theta=10000.0, per_axis=case["per_axis"], interleaved=case["interleaved"],
                          inverse=case["inverse"], seq_major=case["seq_major"],
                          out_seq_major=case["out_seq_major"])
    kw = dict(causal=case["causal"], window=case["window"] or None, softcap=case["softcap"] or None)
    if case["op"] == "lse":
        return mgq.attention_lse(state["q"], state["k"], state["v"], **kw)
    return mgq.attention_backward(state["do"], state["q"], state["k"], state["v"], state["o"],
                                  state["lse"], **kw)


# ---------------------------------------------------------------- work
def _seen_pairs(case):
    """Visible (query, key) pairs of one head."""
    lq, lk = case["q_len"], case["kv_len"]
    pos = np.arange(lq, dtype=np.int64) + (lk - lq)
    hi = np.minimum(pos, lk - 1) if case["causal"] or case["window"] > 0 else np.full(lq, lk - 1)
    lo = np.maximum(pos - case["window"] + 1, 0) if case["window"] > 0 else np.zeros(lq, np.int64)
    return int(np.maximum(hi - lo + 1, 0).sum())


def work(case):
    b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    if case["op"] == "rotary":
        e = 2 if case["dtype"] == "bf16" else 4
        n = b * case["length"] * (hq + hkv)
        axes = len(case["sections"].split(","))
        pairs = sum(int(s) for s in case["sections"].split(","))
        return {"bytes": 2 * e * n * d + 4 * axes * b * case["length"], "flops": 6 * n * pairs}
    q = 2 * b * hq * case["q_len"] * d
    kv = 2 * b * hkv * case["kv_len"] * d
    stat = 4 * b * hq * case["q_len"]
    pairs = b * hq * _seen_pairs(case)
    if case["op"] == "lse":
        return {"bytes": 2 * q + 2 * kv + stat, "flops": 4 * d * pairs}
    return {"bytes": 4 * q + 4 * kv + stat, "flops": 10 * d * pairs}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(st)
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    b, hq, lq, d = q.shape
    hkv, lk = k.shape[1], k.shape[2]
    group = hq // hkv
    query = torch.arange(lq, device=q.device).unsqueeze(1) + lk - lq
    dist = query - torch.arange(lk, device=q.device).unsqueeze(0)
    hide = torch.zeros_like(dist, dtype=torch.bool)
    if case["causal"] or case["window"] > 0:
        hide |= dist < 0
    if case["window"] > 0:
        hide |= dist >= case["window"]
    first, second = torch.zeros_like(q), None
    if case["op"] == "lse":
        second = torch.zeros(b, hq, lq, dtype=torch.float64, device=q.device)
    else:
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
        delta = (st["do"].double() * st["o"].double()).sum(-1)
    for i in range(b):
        for h in range(hq):
            kh, vh = k[i, h // group], v[i, h // group]
            z = torch.einsum("qd,kd->qk", q[i, h], kh) / math.sqrt(d)
            th = torch.tanh(z / case["softcap"]) if case["softcap"] > 0 else None
            if th is not None:
                z = th * case["softcap"]
            z[hide] = -math.inf
            if case["op"] == "lse":
                second[i, h] = torch.logsumexp(z, -1)
                w = torch.exp(z - second[i, h].clamp(min=-1e300).unsqueeze(-1))
                first[i, h] = w @ vh
            else:
                stat = st["lse"][i, h].double().clamp(min=-1e300).unsqueeze(-1)
                w = torch.exp(z - stat)
                gz = w * (torch.einsum("qd,kd->qk", st["do"][i, h].double(), vh)
                          - delta[i, h].unsqueeze(-1))
                if th is not None:
                    gz = gz * (1 - th.square())
                gz = gz / math.sqrt(d)
                first[i, h] = gz @ kh
                dk[i, h // group] += torch.einsum("qk,qd->kd", gz, q[i, h])
                dv[i, h // group] += torch.einsum("qk,qd->kd", w, st["do"][i, h].double())
    return (first, second) if case["op"] == "lse" else (first, dk, dv)


def _exact_rotary(st):
    case, sections = st["case"], st["sections"]
    pairs = sum(sections)
    turn = []
    for a, s in enumerate(sections):
        at = sum(sections[:a])
        for j in range(s):
            f = 10000.0 ** (-(j / s if case["per_axis"] else (at + j) / pairs))
            turn.append(st["positions"][a].double() * f)
    turn = torch.stack(turn, -1) * (-1.0 if case["inverse"] else 1.0)
    unit = torch.polar(torch.ones_like(turn), turn)
    out = []
    for n in ("q", "k"):
        x = st[n].double()
        if not case["seq_major"]:
            x = x.transpose(1, 2)
        y = x.clone()
        if case["interleaved"]:
            re, im = slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)
        else:
            re, im = slice(0, pairs), slice(pairs, 2 * pairs)
        z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * unit.unsqueeze(2)
        y[..., re], y[..., im] = z.real, z.imag
        out.append(y if case["out_seq_major"] else y.transpose(1, 2).contiguous())
    return tuple(out)
