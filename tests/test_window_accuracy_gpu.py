"""Window attention where accuracy and addresses are hardest: logits in the thousands with
their gradients, 32-bit results as a whole, the line of chunks at every head width, graphs
that hold workspaces and changed lengths, caches past 32-bit offsets."""
import math

import pytest
import torch

from structured_attention_video_b200 import (_lib, paged_attention, window_attention,
                                             window_attention_backward)
from window_reference import U, assert_within, attention, visible

pytestmark = pytest.mark.gpu
NAN = float("nan")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(seed, dtype, B, H, Hkv, d, Nq, Nk):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda h, n: torch.randn((B, h, n, d), generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    return r(H, Nq), r(Hkv, Nk), r(Hkv, Nk), r(H, Nq)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    torch.cuda.synchronize()
    return _lib.monarch_last_device_status(None)


def row_bounds(q, k, v, dout, ref, window):
    """Bounds on the errors of out, dq, dk and dv as window_reference derives them, with the
    error of a probability from its own row's largest |q|.|k| instead of the whole call's.
    The backward takes exp(logit - lse) with lse rounded to 32 bits: three roundings of
    numbers as large as |lse| (its own, and the factors ln 2 and log2 e), which 4 2^-24
    |lse| holds."""
    u = U[q.dtype]
    up = max(u, 2.0 ** -24)
    q, k, v, do = (x.double() for x in (q, k, v, dout))
    G = q.shape[1] // k.shape[1]
    k, v = (x.repeat_interleave(G, dim=1) for x in (k, v))
    d = q.shape[3]
    scale = 1 / math.sqrt(d)
    see = visible(q.shape[0], q.shape[2], k.shape[2], window, 0, 1, None, None, q.device)[:, None]
    a = torch.where(see, q @ k.transpose(-1, -2) * scale, -math.inf)
    p = torch.softmax(a, -1)
    mag = torch.where(see, q.abs() @ k.abs().transpose(-1, -2) * scale, 0.0).amax(-1, keepdim=True)
    e = (d + 4) * 2.0 ** -24 * mag + 2.0 ** -21
    n_sum = 2.0 ** -24 * 64
    out = p @ v
    out_err = (up + 2 * e + n_sum) * (p @ v.abs()) * 1.01 + u * out.abs()
    eb = 2 * e + 4 * 2.0 ** -24 * ref["lse"][..., None].abs()
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - (do * out).sum(-1, keepdim=True))
    delta_err = (do.abs() * out_err).sum(-1, keepdim=True)
    dp_err = (d + 4) * 2.0 ** -24 * (do.abs() @ v.abs().transpose(-1, -2))
    ds_err = (up + eb + n_sum) * ds.abs() + p * (1 + eb) * (delta_err + dp_err) * 1.01
    p_err = (up + eb + n_sum) * p * 1.01
    fold = lambda x: x.view(x.shape[0], -1, G, *x.shape[2:]).sum(2)   # noqa: E731
    return {"out": out_err,
            "dq": ds_err @ k.abs() * scale * 1.01 + u * ref["dq"].abs(),
            "dk": fold(ds_err.transpose(-1, -2) @ q.abs()) * scale * 1.01 + u * ref["dk"].abs(),
            "dv": fold(p_err.transpose(-1, -2) @ do.abs()) + u * ref["dv"].abs()}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [(-1, -1), (-1, 0)])
@pytest.mark.parametrize("d,Nq,Nk", [(64, 200, 200), (128, 1, 300), (32, 130, 900)])
def test_large_logits_and_their_gradients(dtype, window, d, Nq, Nk):
    """Logits in the thousands, one key far ahead in most rows."""
    q, k, v, dout = make(31, dtype, 1, 4, 2, d, Nq, Nk)
    q, k = q * 30, k * 30
    ref = attention(q, k, v, dout, window=window)
    assert float(ref["lse"].abs().max()) > 2000
    bound = row_bounds(q, k, v, dout, ref, window)
    out, lse = window_attention(q, k, v, window=window, return_lse=True)
    grads = window_attention_backward(q, k, v, out, lse, dout, window=window)
    assert status() == 0
    assert_within(lse, ref["lse"], ref["lse_bound"], "lse")
    for name, got in zip(("out", "dq", "dk", "dv"), (out, *grads)):
        assert_within(got, ref[name], bound[name], name)


@pytest.mark.parametrize("d,Nq,Nk,window", [(64, 333, 333, (-1, 0)), (128, 200, 3000, (-1, -1)),
                                            (32, 900, 900, (64, 64)), (64, 4, 9000, (-1, 0))])
def test_float32_results_as_a_whole(d, Nq, Nk, window):
    """The norm of the error over the norm of the result.  Roundings are independent and of
    2^-24 / sqrt(3) of the running sum; the running sums of a product of n random terms grow
    like a random walk, which makes 2^-24 0.41 sqrt(n) of the result.  A result passes through
    one sum of d terms with a logit of order one, one of at most n keys or queries, and the
    exponential, division and rounding (8 halves of a step together); the gradients through
    two such chains.  Doubled for what is not quite independent."""
    q, k, v, dout = make(32, "f32", 2, 4, 2, d, Nq, Nk)
    ref = attention(q, k, v, dout, window=window)
    out, lse = window_attention(q, k, v, window=window, return_lse=True)
    grads = window_attention_backward(q, k, v, out, lse, dout, window=window)
    chain = 2.0 ** -24 * (0.5 * math.sqrt(d) + 0.5 * math.sqrt(max(2 * Nq, Nk)) + 8)
    for name, got, chains in zip(("out", "dq", "dk", "dv"), (out, *grads), (1, 2, 2, 2)):
        err = float((got.double() - ref[name]).norm() / ref[name].norm())
        assert err < 2 * chains * chain, (name, err, 2 * chains * chain)


@pytest.mark.parametrize("mask", [((-1, -1), 0, 1), ((-1, 0), 0, 1), ((1500, 0), 40, 1),
                                  ((2, 0), 1, 400)])
def test_line_of_chunks_at_width_32(mask):
    """Heads of 32 columns run in tiles of 64: the line, its parts and their join."""
    window, sinks, frame = mask
    lens = (6000, 0, 4097, 350)
    q, k, v, _ = make(33, "bf16", 4, 3, 1, 32, 600, 6000)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = NAN, NAN
    mask = dict(window=window, sinks=sinks, frame=frame, lengths=ints(*lens))
    ref = attention(q, k, v, **mask)
    out, lse = window_attention(q, k, v, return_lse=True, **mask)
    assert status() == 0
    assert_within(out, ref["out"], ref["out_bound"], "out")
    assert_within(lse, ref["lse"], ref["lse_bound"], "lse")


def test_graph_with_workspaces_and_changed_lengths():
    """One graph that holds a forward over the line of chunks, a call of one token in many
    clusters, the same over pages and a backward with divided key tiles; replayed on other
    inputs and, as a server does, on lengths that have grown and shrunk."""
    Nk, Hkv, d = 20000, 1, 64
    q, k, v, dout = make(34, "bf16", 2, 2, Hkv, d, 300, Nk)
    qs, ks, vs, ds = make(35, "bf16", 1, 4, 1, d, 1000, 1000)
    pages = [x.view(2, Hkv, Nk // 32, 32, d).transpose(1, 2).reshape(-1, Hkv, 32, d).contiguous()
             for x in (k, v)]
    table = torch.arange(2 * Nk // 32, device="cuda", dtype=torch.int32).view(2, -1)
    lengths = ints(20000, 9000)
    kw = dict(window=(-1, 0), lengths=lengths)

    def step():
        out, lse = window_attention(q, k, v, return_lse=True, **kw)
        one = window_attention(q[:, :, :1], k, v, **kw)
        paged = paged_attention(q[:, :, 0], *pages, table, lengths)
        so, sl = window_attention(qs, ks, vs, return_lse=True, starts=0)
        return (out, lse, one, paged, so, sl,
                *window_attention_backward(qs, ks, vs, so, sl, ds, starts=0))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for n in ((20000, 9000), (17, 20000), (0, 301), (19999, 0)):
        for x in (q, qs, ks, vs, ds):
            x.copy_(torch.randn_like(x))
        lengths.copy_(ints(*n))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(captured, step()):
            assert torch.equal(x, y)
        assert torch.equal(captured[2][:, :, 0], captured[3])   # the cache in pages
    ref = attention(q, k, v, **kw)
    assert_within(captured[0], ref["out"], ref["out_bound"], "out")
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_past_32_bit_offsets(dtype):
    """Keys and values in a cache whose last head starts past 2^31 elements, read by the
    forward and by both passes of the backward."""
    cap, Hkv, d = 1 << 21, 9, 128
    q, k, v, dout = make(36, dtype, 1, Hkv, Hkv, d, 130, 200)
    ref = attention(q, k, v, dout)
    cache = torch.empty((2, 1, Hkv, cap, d), dtype=DT[dtype], device="cuda")
    kc, vc = cache[0, :, :, -200:], cache[1, :, :, -200:]
    kc.copy_(k)
    vc.copy_(v)
    out, lse = window_attention(q, kc, vc, return_lse=True)
    grads = window_attention_backward(q, kc, vc, out, lse, dout)
    few = window_attention(q[:, :, -3:], kc, vc)
    assert status() == 0
    assert_within(out, ref["out"], ref["out_bound"], "out")
    assert_within(few, ref["out"][:, :, -3:], ref["out_bound"][:, :, -3:], "few queries")
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert_within(got, ref[name], ref[name + "_bound"], name)


def test_float32_pages_past_32_bit_offsets():
    pages, page, Hkv, d = 70000, 64, 4, 128
    q, k, v, _ = make(37, "f32", 1, 8, Hkv, d, 1, 128)
    pools = torch.empty((2, pages, Hkv, page, d), device="cuda")
    at = [pages - 1, pages - 3]
    for i, pg in enumerate(at):
        for pool, x in zip(pools, (k, v)):
            pool[pg] = x[0, :, i * page:(i + 1) * page]
    ref = attention(q, k, v)
    out = paged_attention(q[:, :, 0], pools[0], pools[1], ints(*at).view(1, 2), ints(128))
    assert status() == 0
    assert_within(out, ref["out"][:, :, 0], ref["out_bound"][:, :, 0], "out")


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("H,Hkv,Nq,Nk", [(3, 3, 6, 3), (12, 3, 1, 241), (2, 1, 70, 70)])
def test_gradients_of_many_short_ragged_sequences(d, H, Hkv, Nq, Nk):
    """Forty sequences of no to a few hundred keys, a block of them without any: many short
    blocks one after another, many times."""
    B = 40
    lens = [(0, 0, Nk, 1, Nk, (7 * b) % (Nk + 1), 0, Nk)[b % 8] for b in range(B)]
    q, k, v, dout = make(38, "bf16", B, H, Hkv, d, Nq, Nk)
    kw = dict(window=(300, -1), sinks=3, lengths=ints(*lens))
    ref = attention(q, k, v, dout, **kw)
    out, lse = window_attention(q, k, v, return_lse=True, **kw)
    first = window_attention_backward(q, k, v, out, lse, dout, **kw)
    for name, got in zip(("dq", "dk", "dv"), first):
        assert_within(got, ref[name], ref[name + "_bound"], name)
    for _ in range(100):
        again = window_attention_backward(q, k, v, out, lse, dout, **kw)
    assert status() == 0
    assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("starts", [2 ** 31 - 1, -2 ** 31 + 1])
def test_float32_blocks_that_see_no_key_drain_their_copies(d, starts):
    """Every row lies outside its sequence, so each block has only its own rows' copies and
    must not end before they do."""
    q, k, v, dout = make(39, "f32", 4, 8, 2, d, 700, 300)
    good = make(40, "f32", 1, 2, 1, d, 200, 200)
    want = window_attention(*good[:3], return_lse=True)
    for _ in range(20):
        out, lse = window_attention(q, k, v, starts=starts, return_lse=True)
        grads = window_attention_backward(q, k, v, out, lse, dout, starts=starts)
        again = window_attention(*good[:3], return_lse=True)
    assert status() == 0
    assert (lse == -math.inf).all()
    assert all((x == 0).all() for x in (out, *grads))
    assert all(torch.equal(x, y) for x, y in zip(want, again))
