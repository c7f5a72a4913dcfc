"""Torch-facing entry points of the rotary positions: argument checks and marshalling
onto the C ABI (monarch_rotary, monarch_rotary_frequencies)."""
from __future__ import annotations

import struct

import torch

from . import _lib
from .window import _device_and_dtype, _index_pointer, _is_bnhd, _launch, _strides

_STYLES = ("interleaved", "half")
_pack_desc = struct.Struct("@16ifPPqq12q").pack   # monarch_rotary_desc
_desc_from = _lib.RotaryDesc.from_buffer_copy
_SCALINGS = {None: _lib.ROTARY_PLAIN, "linear": _lib.ROTARY_LINEAR, "ntk": _lib.ROTARY_NTK,
             "yarn": _lib.ROTARY_YARN}


def rotary_frequencies(dims, *, base=10000.0, scaling=None, factor=1.0, original=0,
                       beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(freqs, magnitude): the float64 frequencies, in radians per position, of axes of
    the given widths (even, in elements: 2 a pair), one after another, and the factor
    for `magnitude` of rotary().  scaling for contexts beyond the trained length: None,
    "linear" (positions divided by factor), "ntk" (a larger base) or "yarn" (by parts;
    original = the trained length)."""
    if scaling not in _SCALINGS:
        raise ValueError("scaling must be one of %s" % (list(_SCALINGS),))
    if isinstance(dims, int):
        dims = (dims,)
    freqs, magnitude = [], 1.0
    for width in dims:
        if width < 0 or width % 2:
            raise ValueError("the width of an axis must be even")
        if width == 0:
            continue
        status, part, magnitude = _lib.monarch_rotary_frequencies(
            width // 2, base, _SCALINGS[scaling], factor, original, beta_fast, beta_slow)
        _lib.check(status, "monarch_rotary_frequencies")
        freqs += part
    return torch.tensor(freqs, dtype=torch.float64, device=device), magnitude


def _run(q, k, freqs, dims, style, grid, positions, start, magnitude, layout, out, inverse):
    bnhd = _is_bnhd(layout)
    if style not in _STYLES:
        raise ValueError("style must be one of %s" % (list(_STYLES),))
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("expected 4-D tensors")
    if out is None:
        q_out = torch.empty_like(q)
        k_out = None if k is None else torch.empty_like(k)
    else:
        q_out, k_out = out
        if (k is None) != (k_out is None):
            raise ValueError("out must be (q_out, k_out), k_out None exactly when k is")
    B, H, N, d = q.shape
    if bnhd:
        H, N = N, H
    if q_out.shape != q.shape or (k is not None and k_out.shape != k.shape):
        raise ValueError("outputs must have the inputs' shapes")
    sq, so = _strides(q, bnhd), _strides(q_out, bnhd)
    if k is None:
        dev, dtype = _device_and_dtype(q, q_out)
        Hkv, sk, sko, kp, kop = 0, (0, 0, 0), (0, 0, 0), None, None
    else:
        dev, dtype = _device_and_dtype(q, q_out, k, k_out)
        kB, Hkv, kN, kd = k.shape
        if bnhd:
            Hkv, kN = kN, Hkv
        if kB != B or kN != N or kd != d:
            raise ValueError("q and k must share batch, tokens and head dimension")
        sk, sko = _strides(k, bnhd), _strides(k_out, bnhd)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    if freqs.dtype is not torch.float64 or freqs.dim() != 1 or freqs.get_device() != dev or \
            not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 vector on the inputs' device")
    pairs = freqs.shape[0]
    if dims is None:
        dims = (2 * pairs,)
    axes = len(dims)
    if not 1 <= axes <= 3 or any(w < 0 or w % 2 for w in dims) or sum(dims) != 2 * pairs:
        raise ValueError("dims must be 1 to 3 even widths that sum to twice the frequencies")
    grid_h = grid_w = 0
    if grid is not None:
        f, grid_h, grid_w = grid
        if f * grid_h * grid_w != N:
            raise ValueError("N = %d but f*h*w = %d" % (N, f * grid_h * grid_w))
        if positions is not None:
            raise ValueError("give grid or positions, not both")
    pos, pos_batch, pos_token = 0, 0, 0
    if positions is not None:
        want = (N,) if axes == 1 else (N, axes)
        if positions.dim() == len(want):
            positions = positions[None]
        if positions.dtype is not torch.int32 or positions.get_device() != dev or \
                tuple(positions.shape[1:]) != want or positions.shape[0] not in (1, B) or \
                (axes > 1 and positions.stride(2) != 1):
            raise ValueError("positions must be int32 [N] or [B, N], with several axes a last "
                             "dimension of them, on the inputs' device")
        pos = positions.data_ptr()
        pos_batch = positions.stride(0) if positions.shape[0] > 1 else 0
        pos_token = positions.stride(1) if N > 1 else 0
    first, starts = 0, 0
    if isinstance(start, int):
        if not -2 ** 31 <= start < 2 ** 31:
            raise ValueError("start out of range")
        first = start
    else:
        starts = _index_pointer(start, "start", B, dev)
    try:
        desc = _desc_from(_pack_desc(
            B, N, H, Hkv, d, pairs, axes, dims[0] // 2, dims[1] // 2 if axes > 1 else 0,
            dims[2] // 2 if axes > 2 else 0, style == "half", inverse, grid_h, grid_w, first, dtype,
            magnitude, starts, pos, pos_batch, pos_token, *sq, *sk, *so, *sko))
    except struct.error as e:
        raise ValueError("an argument is not a number in the library's range: %s" % e) from None
    _launch(dev, _lib.monarch_rotary, "monarch_rotary", desc, q.data_ptr(), kp, freqs.data_ptr(),
            q_out.data_ptr(), kop)
    return q_out, k_out


def rotary(q, k, freqs, *, dims=None, style="interleaved", grid=None, positions=None, start=0,
           magnitude=1.0, layout="bhnd", out=None):
    """(q, k) with rotary positions applied: q [B, H, N, d] and k [B, Hkv, N, d] (or None),
    layout "bnhd" with tokens before heads; float32 or bfloat16.

    freqs: float64 [pairs] on the device (rotary_frequencies); the first 2*pairs elements
    of each head turn, the others are copied.  style: pairs (2i, 2i + 1) ("interleaved")
    or (i, i + pairs) ("half").  dims: widths of up to three axes, in elements, that
    split the pairs; one axis by default.  Positions: `positions` int32 [N] or [B, N] (with
    several axes [.., N, axes]); or one axis from `start` on; or with three axes the
    tokens of grid = (frames, rows, columns) with `start` the first frame.  start is an
    int, or int32 [B] on the device.  out = (q_out, k_out) may be the inputs, or slices
    of a cache."""
    return _run(q, k, freqs, dims, style, grid, positions, start, magnitude, layout, out, False)


def rotary_backward(dq, dk, freqs, *, dims=None, style="interleaved", grid=None, positions=None,
                    start=0, magnitude=1.0, layout="bhnd", out=None):
    """Gradients of rotary()'s inputs from those of its outputs: the rotation by the
    negative angles.  Arguments as rotary()."""
    return _run(dq, dk, freqs, dims, style, grid, positions, start, magnitude, layout, out, True)
