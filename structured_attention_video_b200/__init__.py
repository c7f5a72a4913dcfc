"""Tiled MonarchRT attention forward pass for NVIDIA B200 (sm_100a).

    from structured_attention_video_b200 import monarch_attention
    y = monarch_attention(q, k, v, f=21, h=45, w=80, b1=945, b2=80, tiles=4, iters=1)

q, k, v are contiguous CUDA tensors [B, H, N, d] (float32 or bfloat16) with
N = f*h*w tokens in (frame, row, column) order.  The computation runs in the
CUDA kernels of libmonarch.so (C ABI: include/monarch_attn.h); importing the
attention entry points fails loudly when that library is missing.

Next to it: exact attention over a window of frames with the first frames kept
(window_attention, its backward, and paged_attention for one new token over a paged
cache), and the rotary positions of queries and keys (rotary, rotary_backward), which
the Monarch attention takes as an option (rotary=Rotary(...)).
"""

_MODULES = {
    "monarch_attention": "attention", "workspace_bytes": "attention", "kernel_path": "attention",
    "Rotary": "attention",
    "window_attention": "window", "window_attention_backward": "window",
    "window_attention_path": "window", "paged_attention": "window",
    "rotary": "positions", "rotary_backward": "positions", "rotary_frequencies": "positions",
}
__all__ = list(_MODULES)


def __getattr__(name):
    if name in _MODULES:
        from importlib import import_module
        value = getattr(import_module("." + _MODULES[name], __name__), name)
        globals()[name] = value   # later look-ups are plain attribute reads
        return value
    raise AttributeError(name)
