"""Rotary positions with one or several axes (argument marshalling only).

A head's first ``2 * sum(sections)`` elements form pairs; the first
``sections[0]`` pairs turn with the positions of axis 0, the next
``sections[1]`` with those of axis 1, and so on (one axis: text; two: the rows
and columns of an image's patches; three: time, height and width of video
tokens).  Elements past the last pair pass through.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .backward import _device, _on, _stream_of, _warn_no_graph

IN_SEQ_MAJOR = 0x1
OUT_SEQ_MAJOR = 0x2
IN_F32 = 0x4
OUT_F32 = 0x8
POS_I64 = 0x10
INTERLEAVED = 0x20
PER_AXIS = 0x40
INVERSE = 0x80

_DTYPES = (torch.bfloat16, torch.float32)


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, *, sections,
           theta: float = 10000.0, per_axis: bool = False, interleaved: bool = False,
           inverse: bool = False, seq_major: bool = False, out_seq_major: bool | None = None,
           out_dtype: torch.dtype | None = None, out=None, stream=None):
    """q and k with every pair turned by its axis' position; ``(q_out, k_out)``.

    q and k (None: no keys) are (batch, heads, length, head_dim), the layout
    that ``attention`` reads, or with ``seq_major`` (batch, length, heads,
    head_dim), the layout of a projection and of ``kv_append``'s new tokens;
    bf16 or fp32, the same for both.  The outputs are in the layout that
    ``out_seq_major`` names and of ``out_dtype``, the inputs' by default.
    positions are (axes, batch, length), int32 or int64.  Pair i of the head,
    the j-th of its axis a, turns by position * theta ** (-i / pairs), or with
    ``per_axis`` theta ** (-j / sections[a]).  Pair i is elements (i, i + pairs),
    or with ``interleaved`` (2 i, 2 i + 1).  ``inverse`` turns back, which is also
    the gradient: pass the outputs' gradients for q and k, with the forward's
    output layout and type as the input's.  ``out`` is a (q_out, k_out) pair of
    tensors to write, q and k themselves where type and layout do not change.
    """
    _check("q", q, q)
    if seq_major:
        b, length, hq, d = q.shape
    else:
        b, hq, length, d = q.shape
    hkv = 0
    if k is not None:
        _check("k", k, q)
        if seq_major:
            bk, lk, hkv, dk = k.shape
        else:
            bk, hkv, lk, dk = k.shape
        if bk != b or lk != length or dk != d:
            raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    given = list(sections)
    sections = [int(s) for s in given]
    if sections != given or sections and (max(sections) > 2 ** 31 - 1 or min(sections) < -2 ** 31):
        raise ValueError(f"sections must be whole numbers of 32 bits, got {given}")
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    device = q.device
    if positions.shape != (len(sections), b, length) or positions.device != device \
            or not positions.is_contiguous():
        raise ValueError(f"positions must be contiguous with shape {(len(sections), b, length)} on "
                         f"{device}, got {tuple(positions.shape)} on {positions.device}")
    _warn_no_graph("rotary", q, k)
    if out_seq_major is None:
        out_seq_major = seq_major
    if out_dtype is None:
        out_dtype = q.dtype
    elif out_dtype not in _DTYPES:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    if out is None:
        out = (None, None)
    elif not isinstance(out, (tuple, list)) or len(out) != 2:
        raise TypeError("out must be a pair (q_out, k_out)")
    with _on(stream):
        q_out = _output(out[0], q, (b, length, hq, d) if out_seq_major else (b, hq, length, d),
                        out_dtype)
        if k is not None:
            k_out = _output(out[1], k, (b, length, hkv, d) if out_seq_major
                            else (b, hkv, length, d), out_dtype)
        elif out[1] is not None:
            raise ValueError("out has a k_out, but there is no k")
        else:
            k_out = None
    flags = ((IN_SEQ_MAJOR if seq_major else 0) | (OUT_SEQ_MAJOR if out_seq_major else 0)
             | (IN_F32 if q.dtype == torch.float32 else 0)
             | (OUT_F32 if out_dtype == torch.float32 else 0)
             | (POS_I64 if positions.dtype == torch.int64 else 0)
             | (INTERLEAVED if interleaved else 0) | (PER_AXIS if per_axis else 0)
             | (INVERSE if inverse else 0))
    with _device(device):
        rc = _lib.load().gqa_attn_rotary(
            q.data_ptr(), None if k is None else k.data_ptr(), q_out.data_ptr(),
            None if k is None else k_out.data_ptr(), positions.data_ptr(), b, length, hq, hkv, d,
            len(sections), (ctypes.c_int * len(sections))(*sections), float(theta), flags,
            _stream_of(stream, device))
    _lib.check(rc, "gqa_attn_rotary")
    return q_out, k_out


def _check(name, t, q):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES or t.dtype != q.dtype:
        raise TypeError(f"q and k must both be bfloat16 or float32, got {name} {t.dtype}")
    if t.dim() != 4 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor")
    if t.device != q.device:
        raise ValueError(f"{name} is on {t.device}, q on {q.device}")


def _output(out, like, shape, dtype):
    if out is None:
        if dtype == like.dtype and like.shape == shape:
            return torch.empty_like(like)
        return like.new_empty(shape, dtype=dtype)
    if (not isinstance(out, torch.Tensor) or out.shape != shape or out.dtype != dtype
            or out.device != like.device or not out.is_contiguous()):
        raise ValueError(f"out must hold contiguous {dtype} tensors of shape {shape} on "
                         f"{like.device}")
    return out
