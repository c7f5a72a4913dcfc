"""The operators together, as a rollout and a training step use them, and the rotary
option of the Monarch attention."""
import pytest
import torch

from structured_attention_video_b200 import (Rotary, monarch_attention, paged_attention, rotary,
                                             rotary_backward, rotary_frequencies,
                                             window_attention, window_attention_backward)
from structured_attention_video_b200.attention import (monarch_attention_backward,
                                                       monarch_attention_kv)
from window_reference import assert_within, attention

pytestmark = pytest.mark.gpu


def randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def test_chunks_of_a_rollout_against_the_whole_clip():
    """Frames come in chunks: each chunk's queries and keys are turned at their frame, the
    keys go into the cache, and the chunk attends to the first frame and the two before
    its own.  The whole clip in one call gives the same rows."""
    B, H, h, w, d, frames = 2, 3, 8, 12, 64, 6
    n, N = h * w, 6 * 8 * 12
    dims = (24, 20, 20)
    freqs, _ = rotary_frequencies(dims)
    q, k, v = (randn(i, B, H, N, d) for i in range(3))
    mask = dict(window=(2, 0), sinks=1, frame=n)
    qa, ka = rotary(q, k, freqs, dims=dims, grid=(frames, h, w))
    whole = window_attention(qa, ka, v, **mask)
    ref = attention(qa, ka, v, **mask)
    assert_within(whole, ref["out"], ref["out_bound"], "whole clip")
    cache_k = torch.full((B, H, N, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    cache_v = cache_k.clone()
    at = 0
    for chunk in (3, 1, 2):
        rows = slice(at * n, (at + chunk) * n)
        qc = torch.empty_like(q[:, :, rows])
        rotary(q[:, :, rows], k[:, :, rows], freqs, dims=dims, grid=(chunk, h, w), start=at,
               out=(qc, cache_k[:, :, rows]))
        cache_v[:, :, rows] = v[:, :, rows]
        at += chunk
        lengths = torch.full((B,), at * n, dtype=torch.int32, device="cuda")
        out = window_attention(qc, cache_k, cache_v, lengths=lengths, **mask)
        assert torch.equal(qc, qa[:, :, rows])
        assert_within(out, ref["out"][:, :, rows], ref["out_bound"][:, :, rows], "chunk")


def test_prompt_then_tokens_over_pages():
    """A prompt through the window attention, then single tokens over pages that hold the
    same keys, page by page, while the window gives old pages back."""
    B, H, Hkv, d, page, prompt, total = 2, 8, 2, 128, 16, 150, 190
    freqs, _ = rotary_frequencies(d)
    q, k, v = randn(1, B, H, total, d), randn(2, B, Hkv, total, d), randn(3, B, Hkv, total, d)
    q, k = rotary(q, k, freqs, style="half")
    mask = dict(window=(63, 0), sinks=4)
    ref = attention(q, k, v, **mask)
    out = window_attention(q[:, :, :prompt], k[:, :, :prompt], v[:, :, :prompt], **mask)
    assert_within(out, ref["out"][:, :, :prompt], ref["out_bound"][:, :, :prompt], "prompt")
    width = -(-total // page)
    order = torch.randperm(B * width, generator=torch.Generator().manual_seed(0)).tolist()
    table = torch.tensor(order, dtype=torch.int32).view(B, width).cuda()
    kp = torch.full((B * width, Hkv, page, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    vp = kp.clone()

    def write(j):
        for b in range(B):
            pg = int(table[b, j // page])
            kp[pg, :, j % page], vp[pg, :, j % page] = k[b, :, j], v[b, :, j]
    for j in range(prompt):
        write(j)
    for j in range(prompt, total, 7):
        for jj in range(j, min(j + 7, total)):
            write(jj)
        last = min(j + 6, total - 1)
        gone = (last - 63) // page
        held = table.clone()
        if gone > 1:
            held[:, 1:gone] = -1
        lengths = torch.full((B,), last + 1, dtype=torch.int32, device="cuda")
        out = paged_attention(q[:, :, last], kp, vp, held, lengths, **mask)
        assert_within(out, ref["out"][:, :, last], ref["out_bound"][:, :, last], "token")
        # the same keys in an ordinary cache
        same = window_attention(q[:, :, last:last + 1], k, v, lengths=lengths, **mask)
        assert_within(same[:, :, 0], ref["out"][:, :, last], ref["out_bound"][:, :, last], "cache")


def test_training_step_against_differences():
    """dq of rotary, window attention and back against central differences of the 64-bit
    form along a direction."""
    B, H, N, d = 1, 2, 96, 32
    freqs, _ = rotary_frequencies(d)
    q, k, v, w, dirn = (randn(i, B, H, N, d, dtype=torch.float32) for i in range(5))
    mask = dict(window=(20, 0), sinks=2)
    qa, ka = rotary(q, k, freqs)
    out, lse = window_attention(qa, ka, v, return_lse=True, **mask)
    dq, dk, _ = window_attention_backward(qa, ka, v, out, lse, w, **mask)
    dq, dk = rotary_backward(dq, dk, freqs, out=(dq, dk))

    def loss(qx, kx):
        t = torch.arange(N, device="cuda").double()[:, None] * freqs
        unit = torch.polar(torch.ones_like(t), t)
        turn = lambda x: torch.view_as_real(torch.view_as_complex(   # noqa: E731
            x.unflatten(-1, (d // 2, 2)).contiguous()) * unit).flatten(-2)
        a = turn(qx) @ turn(kx).transpose(-1, -2) * d ** -0.5
        i = torch.arange(N, device="cuda")
        see = (i[None] <= i[:, None]) & ((i[:, None] - i[None] <= 20) | (i[None] < 2))
        p = torch.softmax(a.masked_fill(~see, float("-inf")), -1)
        return ((p @ v.double()) * w.double()).sum()
    e = 1e-4
    for grad, f in ((dq, lambda t: loss(q.double() + t * dirn.double(), k.double())),
                    (dk, lambda t: loss(q.double(), k.double() + t * dirn.double()))):
        slope = float((f(e) - f(-e)) / (2 * e))
        got = float((grad.double() * dirn.double()).sum())
        # differences: error of order e^2; the gradient: float32 roundings of sums of
        # about N d terms of order 1
        assert abs(slope - got) < 1e-3 * max(1.0, abs(slope)), (slope, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_monarch_attention_with_rotary_positions(dtype):
    f, h, w, H = 2, 8, 32, 2
    d, N = 128, f * h * w
    dims = (44, 42, 42)
    freqs, _ = rotary_frequencies(dims)
    q, k, v, dy = (randn(i, 1, H, N, d, dtype=dtype) for i in range(4))
    shape = dict(f=f, h=h, w=w, b1=16, b2=32, tiles=2)
    spec = Rotary(freqs, dims, start=5)
    qa, ka = rotary(q, k, freqs, dims=dims, grid=(f, h, w), start=5)
    assert torch.equal(monarch_attention(q, k, v, rotary=spec, **shape),
                       monarch_attention(qa, ka, v, **shape))
    got = monarch_attention_backward(q, k, v, dy, rotary=spec, **shape)
    dq, dk, dv = monarch_attention_backward(qa, ka, v, dy, **shape)
    dq, dk = rotary_backward(dq, dk, freqs, dims=dims, grid=(f, h, w), start=5)
    for x, y in zip(got, (dq, dk, dv)):
        assert torch.equal(x, y)
    # the newest frame against both, from the unturned tensors
    n = h * w
    kv = dict(fq=1, fk=2, h=h, w=w, b1=8, b1k=16, b2=32)
    assert torch.equal(
        monarch_attention_kv(q[:, :, n:].contiguous(), k, v, rotary=spec, **kv),
        monarch_attention_kv(qa[:, :, n:].contiguous(), ka, v, **kv))
