"""Torch-facing entry points of the rotary positions.  Argument checks and marshalling
onto the C ABI (monarch_rotary) are native (_torch.py): a wrong argument raises
ValueError, a call that the library refuses MonarchError."""
from __future__ import annotations

import torch

from . import _lib
from ._torch import native as _native

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
    int, or int32 [B] on the device.  out = (q_out, k_out) may be the inputs, each in its
    own place, or slices of a cache."""
    return _native.rotary(q, k, freqs, dims, style, grid, positions, start, magnitude, layout,
                          out, False)


def rotary_backward(dq, dk, freqs, *, dims=None, style="interleaved", grid=None, positions=None,
                    start=0, magnitude=1.0, layout="bhnd", out=None):
    """Gradients of rotary()'s inputs from those of its outputs: the rotation by the
    negative angles.  Arguments as rotary()."""
    return _native.rotary(dq, dk, freqs, dims, style, grid, positions, start, magnitude, layout,
                          out, True)
