"""Torch-facing entry points of the exact attention over a window: argument checks and
marshalling onto the C ABI (monarch_window_attn_*, monarch_paged_attn_ws).

The mask, for sequence b of lengths[b] keys and query i at position
p = starts[b] + i (a real row when 0 <= p < lengths[b]; other rows give zeros):
with fq = p // frame and fk = j // frame it sees key j < lengths[b] when
fk <= fq + right (right = -1: no limit) and fk >= fq - left (left = -1: no limit) or
fk < sinks.  window = (left, right).
"""
from __future__ import annotations

import math

import torch

from . import _lib

_DTYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}
_LAYOUTS = ("bhnd", "bnhd")


def _strides(t, head, token, d):
    """(batch, head, token) strides; a dimension of size 1 gets a stride that the
    library accepts, whatever torch says (it is never used)."""
    shape, st = t.shape, t.stride()
    if st[3] != 1:
        raise ValueError("tensors must have stride 1 along the head dimension")
    return (st[0] if shape[0] > 1 else d, st[head] if shape[head] > 1 else d,
            st[token] if shape[token] > 1 else d)


def _fill(strides, values):
    strides.batch, strides.head, strides.token = values


def _index_tensor(x, name, B, device):
    if x.dtype != torch.int32 or x.shape != (B,) or x.device != device or not x.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of [B] on the inputs' device"
                         % name)
    return x.data_ptr()


def _check(q, *ts):
    if not q.is_cuda:
        raise ValueError("all tensors must be on the same CUDA device")
    if q.dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    for t in ts:
        if t.device != q.device:
            raise ValueError("all tensors must be on the same CUDA device")
        if t.dtype != q.dtype:
            raise ValueError("all tensors must share one dtype")


def _mask(desc, q, window, sinks, frame, scale, d):
    left, right = window
    desc.left, desc.right, desc.sinks, desc.frame = left, right, sinks, frame
    desc.scale = 1.0 / math.sqrt(d) if scale is None else scale
    desc.d = d
    desc.dtype = _DTYPES[q.dtype]


def _describe(q, k, v, out, window, sinks, frame, lengths, starts, scale, layout):
    if layout not in _LAYOUTS:
        raise ValueError("layout must be one of %s" % (list(_LAYOUTS),))
    head, token = (1, 2) if layout == "bhnd" else (2, 1)
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape:
        raise ValueError("expected 4-D tensors, k and v alike")
    _check(q, k, v, out)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    B, d = q.shape[0], q.shape[3]
    if k.shape[0] != B or k.shape[3] != d:
        raise ValueError("q, k and v must share batch and head dimension")
    desc = _lib.WindowDesc()
    desc.B, desc.H, desc.Nq = B, q.shape[head], q.shape[token]
    desc.Hkv, desc.Nk = k.shape[head], k.shape[token]
    _mask(desc, q, window, sinks, frame, scale, d)
    if lengths is not None:
        desc.lengths = _index_tensor(lengths, "lengths", B, q.device)
    if starts is None:
        desc.start = _lib.NEWEST
    elif isinstance(starts, int):
        if not -2 ** 31 < starts < 2 ** 31:
            raise ValueError("starts out of range")
        desc.start = starts
    else:
        desc.starts = _index_tensor(starts, "starts", B, q.device)
    _fill(desc.q, _strides(q, head, token, d))
    _fill(desc.k, _strides(k, head, token, d))
    _fill(desc.v, _strides(v, head, token, d))
    _fill(desc.out, _strides(out, head, token, d))
    return desc


def _workspace(need, workspace, device):
    """(pointer, bytes, the tensor that owns them).  None where the call needs none (256),
    or where validation failed (0) and the call itself says why."""
    if need <= 256:
        return None, 0, None
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError("workspace must be on the inputs' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# The handle of torch's current stream on a device: torch.cuda.current_stream() without
# the Stream object (2.2 us a call, a tenth of a short call's host time).
_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream


def _launch(device, call, where, *args):
    """call(*args, stream) on the device's current stream, with the tensors' device
    current for the launch where it is not."""
    index = device.index
    if index == torch.cuda.current_device():
        status = call(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, _stream(index))
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
    float32 [B, H, Nq] (natural logarithm, -inf in rows that see nothing)."""
    if out is None:
        out = torch.empty_like(q)
    desc = _describe(q, k, v, out, window, sinks, frame, lengths, starts, scale, layout)
    lse = None
    if return_lse:
        lse = torch.empty((desc.B, desc.H, desc.Nq), dtype=torch.float32, device=q.device)
    ws, size, _owner = _workspace(_lib.monarch_window_attn_workspace_bytes(desc), workspace,
                                  q.device)
    _launch(q.device, _lib.monarch_window_attn_fwd_ws, "monarch_window_attn_fwd_ws", desc,
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
            lse.data_ptr() if return_lse else None, ws, size)
    return (out, lse) if return_lse else out


def window_attention_path(q, k, v, *, window=(-1, 0), sinks=0, frame=1, scale=None,
                          layout="bhnd") -> int:
    """0 = float32 FMA kernels, 1 = sm_100a tensor-core kernels, 2 = the kernels for few
    query rows, which split the keys."""
    desc = _describe(q, k, v, q, window, sinks, frame, None, None, scale, layout)
    return _lib.monarch_window_attn_path(desc)


def window_attention_backward(q, k, v, out, lse, dout, *, window=(-1, 0), sinks=0, frame=1,
                              lengths=None, starts=None, scale=None, layout="bhnd",
                              workspace=None):
    """Gradients (dq, dk, dv) of a loss whose gradient with respect to
    window_attention(q, k, v, ...) is dout; out and lse come from that call with the
    same arguments.  dk and dv are summed over the query heads that share a key head."""
    desc = _describe(q, k, v, out, window, sinks, frame, lengths, starts, scale, layout)
    _check(q, dout)
    if dout.shape != q.shape:
        raise ValueError("dout must have q's shape")
    if lse.dtype != torch.float32 or lse.shape != (desc.B, desc.H, desc.Nq) or \
            lse.device != q.device or not lse.is_contiguous():
        raise ValueError("lse must be the forward's contiguous float32 [B, H, Nq]")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    head, token = (1, 2) if layout == "bhnd" else (2, 1)
    grads = _lib.WindowGrads()
    for field, t in ((grads.dout, dout), (grads.dq, dq), (grads.dk, dk), (grads.dv, dv)):
        _fill(field, _strides(t, head, token, desc.d))
    need = max(257, _lib.monarch_window_attn_bwd_workspace_bytes(desc))   # always used
    ws, size, _owner = _workspace(need, workspace, q.device)
    _launch(q.device, _lib.monarch_window_attn_bwd_ws, "monarch_window_attn_bwd_ws", desc, grads,
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
    if q.dim() != 3 or k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        raise ValueError("expected q [B, H, d] and 4-D pools of pages, k and v alike")
    if layout not in _LAYOUTS:
        raise ValueError("layout must be one of %s" % (list(_LAYOUTS),))
    if out is None:
        out = torch.empty_like(q)
    _check(q, k_pages, v_pages, out)
    B, H, d = q.shape
    head, token = (1, 2) if layout == "bhnd" else (2, 1)
    if out.shape != q.shape or k_pages.shape[3] != d:
        raise ValueError("out must have q's shape, and the pages its head dimension")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != B or \
            page_table.device != q.device or page_table.stride(1) != 1:
        raise ValueError("page_table must be int32 [B, width] on the inputs' device")
    page, width = k_pages.shape[token], page_table.shape[1]
    if width < 1 or width * page > 2 ** 30:
        raise ValueError("page table of %d pages of %d keys: out of range" % (width, page))
    desc = _lib.WindowDesc()
    desc.B, desc.H, desc.Hkv, desc.Nq, desc.Nk = B, H, k_pages.shape[head], 1, width * page
    _mask(desc, q, window, sinks, frame, scale, d)
    desc.start = _lib.NEWEST
    desc.lengths = _index_tensor(lengths, "lengths", B, q.device)
    for field, t in ((desc.q, q), (desc.out, out)):
        if t.stride(2) != 1:
            raise ValueError("tensors must have stride 1 along the head dimension")
        _fill(field, (t.stride(0) if B > 1 else d, t.stride(1) if H > 1 else d, d))
    _fill(desc.k, _strides(k_pages, head, token, d))
    _fill(desc.v, _strides(v_pages, head, token, d))
    lse = torch.empty((B, H, 1), dtype=torch.float32, device=q.device) if return_lse else None
    ws, size, _owner = _workspace(_lib.monarch_paged_attn_workspace_bytes(desc), workspace,
                                  q.device)
    _launch(q.device, _lib.monarch_paged_attn_ws, "monarch_paged_attn_ws", desc, q.data_ptr(),
            k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
            page_table.stride(0) if B > 1 else width, page, k_pages.shape[0], out.data_ptr(),
            lse.data_ptr() if return_lse else None, ws, size)
    return (out, lse) if return_lse else out
