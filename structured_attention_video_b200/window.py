"""Torch-facing entry points of the exact attention over a window.  Argument checks and
marshalling onto the C ABI (monarch_window_attn_*, monarch_paged_attn_ws) are native
(_torch.py): a wrong argument raises ValueError, a call that the library refuses
MonarchError.

The mask, for sequence b of lengths[b] keys and query i at position
p = starts[b] + i (a real row when 0 <= p < lengths[b]; other rows give zeros):
with fq = p // frame and fk = j // frame it sees key j < lengths[b] when
fk <= fq + right (right = -1: no limit) and fk >= fq - left (left = -1: no limit) or
fk < sinks.  window = (left, right).
"""
from __future__ import annotations

from ._torch import native as _native


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
    return _native.window_attention(q, k, v, window, sinks, frame, lengths, starts, scale, layout,
                                    out, return_lse, workspace)


def window_attention_path(q, k, v, *, window=(-1, 0), sinks=0, frame=1, scale=None,
                          layout="bhnd") -> int:
    """0 = float32 FMA kernels, 1 = sm_100a tensor-core kernels, 2 = the kernels for few
    query rows, which split the keys."""
    return _native.window_attention_path(q, k, v, window, sinks, frame, None, None, scale, layout)


def window_attention_backward(q, k, v, out, lse, dout, *, window=(-1, 0), sinks=0, frame=1,
                              lengths=None, starts=None, scale=None, layout="bhnd",
                              workspace=None):
    """Gradients (dq, dk, dv) of a loss whose gradient with respect to
    window_attention(q, k, v, ...) is dout; out and lse come from that call with the
    same arguments.  dk and dv are summed over the query heads that share a key head."""
    return _native.window_attention_backward(q, k, v, window, sinks, frame, lengths, starts, scale,
                                             layout, out, lse, dout, workspace)


def paged_attention(q, k_pages, v_pages, page_table, lengths, *, window=(-1, 0), sinks=0,
                    frame=1, scale=None, layout="bhnd", out=None, return_lse=False,
                    workspace=None):
    """One new token a sequence over a paged cache: q [B, H, d], the newest token of
    sequences of lengths[b] keys (int32 [B] on the device, the new one included).

    k_pages and v_pages [pages, Hkv, page, d] (layout "bnhd": [pages, page, Hkv, d]),
    page a power of two from 8 on; page_table int32 [B, width] on the device: key j of
    sequence b is row j % page of page page_table[b, j // page].  Entries whose pages hold
    no visible key are not read.  An entry that is read and lies outside the pool is
    reported by monarch_last_device_status, and its keys count as absent.  Mask, out and
    workspace as window_attention.  A sequence of length 0 gives zeros."""
    return _native.paged_attention(q, k_pages, v_pages, page_table, lengths, window, sinks, frame,
                                   scale, layout, out, return_lse, workspace)
