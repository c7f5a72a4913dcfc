"""Torch-facing entry points of the rotary positions: argument checks and marshalling
onto the C ABI (monarch_rotary, monarch_rotary_frequencies)."""
from __future__ import annotations

import torch

from . import _lib
from .window import _DTYPES, _LAYOUTS, _check, _fill, _index_tensor, _launch, _strides

_STYLES = ("interleaved", "half")
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
    if layout not in _LAYOUTS or style not in _STYLES:
        raise ValueError("layout must be one of %s and style one of %s"
                         % (list(_LAYOUTS), list(_STYLES)))
    head, token = (1, 2) if layout == "bhnd" else (2, 1)
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("expected 4-D tensors")
    if out is None:
        q_out = torch.empty_like(q)
        k_out = None if k is None else torch.empty_like(k)
    else:
        q_out, k_out = out
        if (k is None) != (k_out is None):
            raise ValueError("out must be (q_out, k_out), k_out None exactly when k is")
    _check(q, q_out, *(() if k is None else (k, k_out)))
    B, N, d = q.shape[0], q.shape[token], q.shape[3]
    if q_out.shape != q.shape or (k is not None and k_out.shape != k.shape):
        raise ValueError("outputs must have the inputs' shapes")
    if k is not None and (k.shape[0] != B or k.shape[token] != N or k.shape[3] != d):
        raise ValueError("q and k must share batch, tokens and head dimension")
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or freqs.device != q.device or \
            not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 vector on the inputs' device")
    desc = _lib.RotaryDesc()
    desc.B, desc.N, desc.H, desc.d = B, N, q.shape[head], d
    desc.Hkv = 0 if k is None else k.shape[head]
    pairs = desc.pairs = freqs.shape[0]
    if dims is None:
        dims = (2 * pairs,)
    if not 1 <= len(dims) <= 3 or any(w < 0 or w % 2 for w in dims) or sum(dims) != 2 * pairs:
        raise ValueError("dims must be 1 to 3 even widths that sum to twice the frequencies")
    desc.axes = len(dims)
    for i, w in enumerate(dims):
        desc.pairs_of_axis[i] = w // 2
    desc.half, desc.inverse = int(style == "half"), int(inverse)
    desc.dtype, desc.magnitude = _DTYPES[q.dtype], magnitude
    if grid is not None:
        f, h, w = grid
        if f * h * w != N:
            raise ValueError("N = %d but f*h*w = %d" % (N, f * h * w))
        if positions is not None:
            raise ValueError("give grid or positions, not both")
        desc.grid_h, desc.grid_w = h, w
    if positions is not None:
        want = (N,) if len(dims) == 1 else (N, len(dims))
        if positions.dim() == len(want):
            positions = positions[None]
        if positions.dtype != torch.int32 or positions.device != q.device or \
                tuple(positions.shape[1:]) != want or positions.shape[0] not in (1, B) or \
                (len(want) == 2 and len(dims) > 1 and positions.stride(2) != 1):
            raise ValueError("positions must be int32 [N] or [B, N], with several axes a last "
                             "dimension of them, on the inputs' device")
        desc.positions = positions.data_ptr()
        desc.pos_batch = positions.stride(0) if positions.shape[0] > 1 else 0
        desc.pos_token = positions.stride(1) if N > 1 else 0
    if isinstance(start, int):
        if not -2 ** 31 <= start < 2 ** 31:
            raise ValueError("start out of range")
        desc.start = start
    else:
        desc.starts = _index_tensor(start, "start", B, q.device)
    _fill(desc.q, _strides(q, head, token, d))
    _fill(desc.q_out, _strides(q_out, head, token, d))
    if k is not None:
        _fill(desc.k, _strides(k, head, token, d))
        _fill(desc.k_out, _strides(k_out, head, token, d))
    _launch(q.device, _lib.monarch_rotary, "monarch_rotary", desc, q.data_ptr(),
            None if k is None else k.data_ptr(), freqs.data_ptr(), q_out.data_ptr(),
            None if k is None else k_out.data_ptr())
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
