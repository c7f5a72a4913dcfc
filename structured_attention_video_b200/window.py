"""Torch-facing entry points of the exact attention over a window: argument checks and
marshalling onto the C ABI (monarch_window_attn_*, monarch_paged_attn_ws).

The mask, for sequence b of lengths[b] keys and query i at position
p = starts[b] + i (a real row when 0 <= p < lengths[b]; other rows give zeros):
with fq = p // frame and fk = j // frame it sees key j < lengths[b] when
fk <= fq + right (right = -1: no limit) and fk >= fq - left (left = -1: no limit) or
fk < sinks.  window = (left, right).
"""
from __future__ import annotations

import struct

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}
_LAYOUTS = ("bhnd", "bnhd")

# The structs of the C ABI are packed in one go: a short call's host time is a dozen
# microseconds, and setting their fields one by one is a third of that.
_pack_desc = struct.Struct("@11iifPP12q").pack     # monarch_window_desc
_pack_grads = struct.Struct("@12q").pack           # monarch_window_grads
_desc_from = _lib.WindowDesc.from_buffer_copy
_grads_from = _lib.WindowGrads.from_buffer_copy


def _strides(t, bnhd):
    """(batch, head, token) strides of a 4-D tensor; a dimension of size 1 gets a stride
    that the library accepts, whatever torch says (it is never used)."""
    n0, n1, n2, d = t.shape
    s0, s1, s2, sd = t.stride()
    if sd != 1:
        raise ValueError("tensors must have stride 1 along the head dimension")
    if n0 == 1:
        s0 = d
    if n1 == 1:
        s1 = d
    if n2 == 1:
        s2 = d
    return (s0, s2, s1) if bnhd else (s0, s1, s2)


def _index_pointer(x, name, B, dev):
    if x.dtype is not torch.int32 or x.get_device() != dev or x.dim() != 1 or \
            x.shape[0] != B or not x.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of [B] on the inputs' device"
                         % name)
    return x.data_ptr()


def _device_and_dtype(q, *ts):
    """The device index and the library's dtype code that all tensors share."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("all tensors must be on the same CUDA device")
    dtype = q.dtype
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError("dtype must be float32 or bfloat16")
    for t in ts:
        if t.get_device() != dev:
            raise ValueError("all tensors must be on the same CUDA device")
        if t.dtype is not dtype:
            raise ValueError("all tensors must share one dtype")
    return dev, code


def _is_bnhd(layout):
    if layout not in _LAYOUTS:
        raise ValueError("layout must be one of %s" % (list(_LAYOUTS),))
    return layout == "bnhd"


def _describe(q, k, v, out, window, sinks, frame, lengths, starts, scale, layout):
    """(monarch_window_desc, (B, H, Nq), device index)."""
    bnhd = _is_bnhd(layout)
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape:
        raise ValueError("expected 4-D tensors, k and v alike")
    dev, dtype = _device_and_dtype(q, k, v, out)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    B, H, Nq, d = q.shape
    kB, Hkv, Nk, kd = k.shape
    if bnhd:
        H, Nq, Hkv, Nk = Nq, H, Nk, Hkv
    if kB != B or kd != d:
        raise ValueError("q, k and v must share batch and head dimension")
    start, starts_ptr = 0, 0
    if starts is None:
        start = _lib.NEWEST
    elif isinstance(starts, int):
        if not -2 ** 31 < starts < 2 ** 31:
            raise ValueError("starts out of range")
        start = starts
    else:
        starts_ptr = _index_pointer(starts, "starts", B, dev)
    left, right = window
    try:
        desc = _desc_from(_pack_desc(
            B, H, Hkv, Nq, Nk, d, frame, left, right, sinks, start, dtype,
            d ** -0.5 if scale is None and d else scale or 0.0,
            0 if lengths is None else _index_pointer(lengths, "lengths", B, dev), starts_ptr,
            *_strides(q, bnhd), *_strides(k, bnhd), *_strides(v, bnhd), *_strides(out, bnhd)))
    except struct.error as e:
        raise ValueError("an argument is not a number in the library's range: %s" % e) from None
    return desc, (B, H, Nq), dev


def _workspace(need, workspace, q):
    """(pointer, bytes, the tensor that owns them).  None where the call needs none (256),
    or where validation failed (0) and the call itself says why."""
    if need <= 256:
        return None, 0, None
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != q.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the inputs' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# The handle of torch's current stream on a device: torch.cuda.current_stream() without
# the Stream object (2.2 us a call, a tenth of a short call's host time).
_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(dev, call, where, *args):
    """call(*args, stream) on the device's current stream, with the tensors' device
    current for the launch where it is not."""
    if dev == _current_device():
        status = call(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            status = call(*args, _stream(dev))
    if status:
        _lib.check(status, where)


def window_attention(q, k, v, *, window=(-1, 0), sinks=0, frame=1, lengths=None, starts=None,
                     scale=None, layout="bhnd", out=None, return_lse=False, workspace=None):
    """Exact softmax attention of q [B, H, Nq, d] over k and v [B, Hkv, Nk, d] (layout
    "bnhd": [B, Nq, H, d] and so on) under the window's mask (module docstring).

    H is a multiple of Hkv; d is 32, 64 or 128; float32 or bfloat16.  Strides other than
    the head dimension's are free (multiples of 16 bytes), so slices of a fused
    projection or of a longer cache need no copy.  lengths (int32 [B] on the device)
    gives each sequence's keys, Nk by default; starts (an int or int32 [B] on the
    device) the position of its first query, by default such that the queries are its
    newest tokens.  scale defaults to 1/sqrt(d).  Returns out, or (out, lse) with lse
    float32 [B, H, Nq] (natural logarithm, -inf in rows that see nothing).  out may be a
    strided view that overlaps no input; a workspace (uint8, any size) spares the
    allocation where it is large enough, and calls that overlap must not share one."""
    if out is None:
        out = torch.empty_like(q)
    elif out.data_ptr() in (q.data_ptr(), k.data_ptr(), v.data_ptr()):
        raise ValueError("out must not be an input")
    desc, shape, dev = _describe(q, k, v, out, window, sinks, frame, lengths, starts, scale, layout)
    lse = torch.empty(shape, dtype=torch.float32, device=q.device) if return_lse else None
    ws, size, _owner = _workspace(_lib.monarch_window_attn_workspace_bytes(desc), workspace, q)
    _launch(dev, _lib.monarch_window_attn_fwd_ws, "monarch_window_attn_fwd_ws", desc,
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
            lse.data_ptr() if return_lse else None, ws, size)
    return (out, lse) if return_lse else out


def window_attention_path(q, k, v, *, window=(-1, 0), sinks=0, frame=1, scale=None,
                          layout="bhnd") -> int:
    """0 = float32 FMA kernels, 1 = sm_100a tensor-core kernels, 2 = the kernels for few
    query rows, which split the keys."""
    desc, _, _ = _describe(q, k, v, q, window, sinks, frame, None, None, scale, layout)
    return _lib.monarch_window_attn_path(desc)


def window_attention_backward(q, k, v, out, lse, dout, *, window=(-1, 0), sinks=0, frame=1,
                              lengths=None, starts=None, scale=None, layout="bhnd",
                              workspace=None):
    """Gradients (dq, dk, dv) of a loss whose gradient with respect to
    window_attention(q, k, v, ...) is dout; out and lse come from that call with the
    same arguments.  dk and dv are summed over the query heads that share a key head."""
    desc, shape, dev = _describe(q, k, v, out, window, sinks, frame, lengths, starts, scale, layout)
    _device_and_dtype(q, dout)
    if dout.shape != q.shape:
        raise ValueError("dout must have q's shape")
    if lse.dtype is not torch.float32 or lse.shape != shape or lse.get_device() != dev or \
            not lse.is_contiguous():
        raise ValueError("lse must be the forward's contiguous float32 [B, H, Nq]")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    bnhd = layout == "bnhd"
    grads = _grads_from(_pack_grads(*_strides(dout, bnhd), *_strides(dq, bnhd),
                                    *_strides(dk, bnhd), *_strides(dv, bnhd)))
    need = max(257, _lib.monarch_window_attn_bwd_workspace_bytes(desc))   # always used
    ws, size, _owner = _workspace(need, workspace, q)
    _launch(dev, _lib.monarch_window_attn_bwd_ws, "monarch_window_attn_bwd_ws", desc, grads,
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
            dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws, size)
    return dq, dk, dv


def paged_attention(q, k_pages, v_pages, page_table, lengths, *, window=(-1, 0), sinks=0,
                    frame=1, scale=None, layout="bhnd", out=None, return_lse=False,
                    workspace=None):
    """One new token a sequence over a paged cache: q [B, H, d], the newest token of
    sequences of lengths[b] keys (int32 [B] on the device, the new one included).

    k_pages and v_pages [pages, Hkv, page, d] (layout "bnhd": [pages, page, Hkv, d]),
    page a power of two from 8 on; page_table int32 [B, width] on the device: key j of
    sequence b is row j % page of page page_table[b, j // page].  Entries whose pages hold
    no visible key are not read.  An entry that is read and lies outside the pool is
    reported by monarch_last_device_status, and its keys count as absent.  Mask as
    window_attention.  A sequence of length 0 gives zeros."""
    bnhd = _is_bnhd(layout)
    if q.dim() != 3 or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise ValueError("expected q [B, H, d] and 4-D pools of pages, k and v alike")
    if out is None:
        out = torch.empty_like(q)
    elif out.data_ptr() == q.data_ptr():
        raise ValueError("out must not be an input")
    dev, dtype = _device_and_dtype(q, k_pages, v_pages, out)
    B, H, d = q.shape
    pages, Hkv, page, kd = k_pages.shape
    if bnhd:
        Hkv, page = page, Hkv
    if out.shape != q.shape or kd != d:
        raise ValueError("out must have q's shape, and the pages its head dimension")
    if page_table.dtype is not torch.int32 or page_table.get_device() != dev or \
            page_table.dim() != 2 or page_table.shape[0] != B or page_table.stride(1) != 1:
        raise ValueError("page_table must be int32 [B, width] on the inputs' device")
    width = page_table.shape[1]
    if width < 1 or width * page > 2 ** 30:
        raise ValueError("page table of %d pages of %d keys: out of range" % (width, page))
    qs, os = q.stride(), out.stride()
    if qs[2] != 1 or os[2] != 1:
        raise ValueError("tensors must have stride 1 along the head dimension")
    left, right = window
    try:
        desc = _desc_from(_pack_desc(
            B, H, Hkv, 1, width * page, d, frame, left, right, sinks, _lib.NEWEST, dtype,
            d ** -0.5 if scale is None and d else scale or 0.0,
            _index_pointer(lengths, "lengths", B, dev), 0,
            qs[0] if B > 1 else d, qs[1] if H > 1 else d, d,
            *_strides(k_pages, bnhd), *_strides(v_pages, bnhd),
            os[0] if B > 1 else d, os[1] if H > 1 else d, d))
    except struct.error as e:
        raise ValueError("an argument is not a number in the library's range: %s" % e) from None
    lse = torch.empty((B, H, 1), dtype=torch.float32, device=q.device) if return_lse else None
    ws, size, _owner = _workspace(_lib.monarch_paged_attn_workspace_bytes(desc), workspace, q)
    _launch(dev, _lib.monarch_paged_attn_ws, "monarch_paged_attn_ws", desc, q.data_ptr(),
            k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
            page_table.stride(0) if B > 1 else width, page, pages, out.data_ptr(),
            lse.data_ptr() if return_lse else None, ws, size)
    return (out, lse) if return_lse else out
