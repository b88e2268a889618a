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
from .backward import _device, _on, _stream_of

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
    tensors = [("q", q)] + ([] if k is None else [("k", k)])
    for n, t in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
        if t.dtype not in _DTYPES or t.dtype != q.dtype:
            raise TypeError(f"q and k must both be bfloat16 or float32, got {n} {t.dtype}")
        if t.dim() != 4 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous 4-D CUDA tensor")
        if t.device != q.device:
            raise ValueError(f"{n} is on {t.device}, q on {q.device}")
    hd, ld = (2, 1) if seq_major else (1, 2)
    b, length, hq, d = q.shape[0], q.shape[ld], q.shape[hd], q.shape[3]
    hkv = 0 if k is None else k.shape[hd]
    if k is not None and (k.shape[0], k.shape[ld], k.shape[3]) != (b, length, d):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    sections = [int(s) for s in sections]
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    if tuple(positions.shape) != (len(sections), b, length) or positions.device != q.device \
            or not positions.is_contiguous():
        raise ValueError(f"positions must be contiguous with shape {(len(sections), b, length)} on "
                         f"{q.device}, got {tuple(positions.shape)} on {positions.device}")
    if out_seq_major is None:
        out_seq_major = seq_major
    if out_dtype is None:
        out_dtype = q.dtype
    if out_dtype not in _DTYPES:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    if out is not None and (not isinstance(out, (tuple, list)) or len(out) != 2):
        raise TypeError("out must be a pair (q_out, k_out)")
    outs = []
    for i, (t, heads) in enumerate(((q, hq), (k, hkv))):
        o = None if out is None else out[i]
        if t is None:
            if o is not None:
                raise ValueError("out has a k_out, but there is no k")
        else:
            shape = (b, length, heads, d) if out_seq_major else (b, heads, length, d)
            if o is None:
                with _on(stream):
                    o = torch.empty(shape, dtype=out_dtype, device=q.device)
            elif (not isinstance(o, torch.Tensor) or tuple(o.shape) != shape
                  or o.dtype != out_dtype or o.device != q.device or not o.is_contiguous()):
                raise ValueError(f"out must hold contiguous {out_dtype} tensors of shape {shape} on "
                                 f"{q.device}")
        outs.append(o)
    flags = ((IN_SEQ_MAJOR if seq_major else 0) | (OUT_SEQ_MAJOR if out_seq_major else 0)
             | (IN_F32 if q.dtype == torch.float32 else 0)
             | (OUT_F32 if out_dtype == torch.float32 else 0)
             | (POS_I64 if positions.dtype == torch.int64 else 0)
             | (INTERLEAVED if interleaved else 0) | (PER_AXIS if per_axis else 0)
             | (INVERSE if inverse else 0))
    ptr = [None if t is None else t.data_ptr() for t in (q, k, *outs)]
    with _device(q.device):
        rc = _lib.load().gqa_attn_rotary(*ptr, positions.data_ptr(), b, length, hq, hkv, d,
                                         len(sections), (ctypes.c_int * len(sections))(*sections),
                                         float(theta), flags, _stream_of(stream, q.device))
    _lib.check(rc, "gqa_attn_rotary")
    return tuple(outs)
