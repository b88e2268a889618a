"""The training forward and the backward pass (argument marshalling only).

``attention_lse`` is ``attention`` that also returns every row's log-sum-exp,
fp32 (batch, num_q_heads, q_len), natural logarithm, -inf for a row without
a visible key.  ``attention_backward`` takes it, the output and the output's
gradient, recomputes the probabilities and returns the gradients of q, k and
v.  Results over disjoint sets of keys merge by the same statistic:
``lse = logsumexp_s lse_s``, ``o = sum_s exp(lse_s - lse) o_s``.

Neither these functions nor ``rotary`` record an autograd graph: a training
step calls the backward functions itself, in an ``autograd.Function`` or under
``torch.no_grad()``.  Called with tensors that require a gradient while
gradients are recorded they warn, since ``loss.backward()`` stops there.
"""
from __future__ import annotations

import contextlib
import ctypes
import warnings

import torch

from . import _lib
from .attention import _args, _check_tensor


def _stream_of(stream, device) -> int:
    """The cudaStream_t of ``stream``, or of ``device``'s current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream


def _device(device):
    """``device`` as the current one; entering it costs more than asking."""
    if torch.cuda.current_device() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _on(stream):
    """Allocations for work on ``stream`` belong to that stream: their memory
    is then reused only after the work, whatever the current stream is."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _warn_no_graph(name, *tensors):
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            warnings.warn(f"{name} records no autograd graph: gradients stop at its results, and its "
                          "inputs require one (call it in an autograd.Function or under "
                          "torch.no_grad())", stacklevel=3)
            return


def _check_qkv(q, k, v):
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(n, t)
        if not t.is_cuda:
            raise ValueError(f"{n} must be a CUDA tensor")
        if t.device != q.device:
            raise ValueError(f"{n} is on {t.device}, q on {q.device}")
    b, hq, lq, d = q.shape
    if v.shape != k.shape or k.shape[0] != b or k.shape[3] != d:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, "
                         f"v {tuple(v.shape)}")
    return b, lq, k.shape[2], hq, k.shape[1], d


def _check_like(name, t, q):
    _check_tensor(name, t)
    if t.shape != q.shape or t.device != q.device:
        raise ValueError(f"{name} must have shape {tuple(q.shape)} on {q.device}, got "
                         f"{tuple(t.shape)} on {t.device}")


def _check_rows(name, t, q):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if t.shape != q.shape[:3] or t.device != q.device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(q.shape[:3])} on {q.device}")


def attention_lse(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False,
                  window: int | None = None, softcap: float | None = None,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Masked GQA attention forward and its rows' log-sum-exp: ``(o, lse)``."""
    dims = _check_qkv(q, k, v)
    _warn_no_graph("attention_lse", q, k, v)
    with _on(stream):
        if out is None:
            out = torch.empty_like(q)
        else:
            _check_like("out", out, q)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        else:
            _check_rows("lse", lse, q)
    lib = _lib.load()
    with _device(q.device):
        rc = lib.gqa_attn_fwd_lse(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  lse.data_ptr(), *dims, *_args(window, softcap, causal),
                                  _stream_of(stream, q.device))
    _lib.check(rc, "gqa_attn_fwd_lse")
    return out, lse


def attention_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       o: torch.Tensor, lse: torch.Tensor, *, dlse: torch.Tensor | None = None,
                       causal: bool = False, window: int | None = None,
                       softcap: float | None = None, dq: torch.Tensor | None = None,
                       dk: torch.Tensor | None = None, dv: torch.Tensor | None = None,
                       stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients ``(dq, dk, dv)`` of ``attention_lse(q, k, v)`` given the
    gradients ``do`` of its output ``o`` and, optionally, ``dlse`` of its
    ``lse``; the mask options are those of the forward call."""
    dims = _check_qkv(q, k, v)
    _check_like("do", do, q)
    _check_like("o", o, q)
    _check_rows("lse", lse, q)
    if dlse is not None:
        _check_rows("dlse", dlse, q)
    _warn_no_graph("attention_backward", do, q, k, v, o, lse, dlse)
    c, w, s = _args(window, softcap, causal)
    lib = _lib.load()
    size = ctypes.c_size_t(0)
    _lib.check(lib.gqa_attn_bwd_scratch(*dims, c, w, ctypes.byref(size)), "gqa_attn_bwd_scratch")
    with _on(stream):
        outs = []
        for n, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            if t is None:
                t = torch.empty_like(like)
            else:
                _check_like(n, t, like)
            outs.append(t)
        scratch = torch.empty(size.value, dtype=torch.uint8, device=q.device)
    with _device(q.device):
        rc = lib.gqa_attn_bwd(do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                              o.data_ptr(), lse.data_ptr(),
                              None if dlse is None else dlse.data_ptr(),
                              *[t.data_ptr() for t in outs], scratch.data_ptr(), size.value,
                              *dims, c, w, s, _stream_of(stream, q.device))
    _lib.check(rc, "gqa_attn_bwd")
    return tuple(outs)
