"""Window attention, forward and backward, and paged attention against the plain 64-bit
form: types, head layouts, lengths from one token on, odd sizes, strides, masks that
leave rows empty, garbage where nothing may be read."""
import pytest
import torch

from structured_attention_video_b200 import (_lib, paged_attention, window_attention,
                                             window_attention_backward, window_attention_path)
from window_reference import assert_within, attention

pytestmark = pytest.mark.gpu
NAN = float("nan")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(seed, dtype, B, H, Hkv, d, Nq, Nk, layout="bhnd"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda h, n: torch.randn((B, h, n, d) if layout == "bhnd" else (B, n, h, d),  # noqa: E731
                                 generator=g, device="cuda").to(DT[dtype])
    return r(H, Nq), r(Hkv, Nk), r(Hkv, Nk), r(H, Nq)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(q, k, v, dout=None, layout="bhnd", **mask):
    ref = attention(q, k, v, dout, layout=layout, **mask)
    out, lse = window_attention(q, k, v, layout=layout, return_lse=True, **mask)
    torch.cuda.synchronize()
    _lib.check(_lib.monarch_last_device_status(None), "device status")
    assert_within(out, ref["out"], ref["out_bound"], "out")
    assert_within(lse, ref["lse"], ref["lse_bound"], "lse")
    if dout is not None:
        grads = window_attention_backward(q, k, v, out, lse, dout, layout=layout, **mask)
        torch.cuda.synchronize()
        _lib.check(_lib.monarch_last_device_status(None), "device status")
        for name, got in zip(("dq", "dk", "dv"), grads):
            assert_within(got, ref[name], ref[name + "_bound"], name)
    return out, lse


# (window, sinks, frame)
MASKS = [((-1, 0), 0, 1), ((-1, -1), 0, 1), ((5, 0), 2, 1), ((64, 64), 0, 1), ((0, 0), 0, 1),
         ((1, 0), 1, 30), ((0, 2), 1, 64), ((127, 0), 4, 1)]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 64)])
def test_self_attention_masks(dtype, d, mask):
    window, sinks, frame = mask
    q, k, v, dout = make(1, dtype, 2, 4, 2, d, 333, 333)
    check(q, k, v, dout, window=window, sinks=sinks, frame=frame, starts=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 2, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 385])
def test_lengths(dtype, N):
    q, k, v, dout = make(N, dtype, 1, 2, 1, 64 if N % 2 else 128, N, N)
    check(q, k, v, dout, window=(-1, 0))
    check(q, k, v, dout, window=(70, 3), sinks=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (5, 1), (6, 3), (16, 2)])
def test_heads(dtype, d, H, Hkv):
    q, k, v, dout = make(3, dtype, 2, H, Hkv, d, 150, 150, "bnhd")
    check(q, k, v, dout, layout="bnhd", window=(40, 0), sinks=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq", [1, 3, 16, 65, 130, 300])
def test_new_tokens_against_a_cache_with_garbage_behind(dtype, Nq):
    B, Nk = 3, 700
    q, k, v, _ = make(4, dtype, B, 4, 2, 128, Nq, Nk)
    lengths = ints(700, 301, 0)     # the last sequence holds nothing: its rows are zeros
    for b, n in enumerate((700, 301, 0)):
        k[b, :, n:], v[b, :, n:] = NAN, NAN
    for window, sinks in (((-1, 0), 0), ((100, 0), 5), ((-1, -1), 0), ((31, 2), 70)):
        out, lse = check(q, k, v, window=window, sinks=sinks, lengths=lengths)
        assert (out[2] == 0).all() and (lse[2] == -float("inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_training_batch_with_garbage_in_the_padding(dtype):
    B, N = 4, 270
    q, k, v, dout = make(5, dtype, B, 4, 2, 64, N, N)
    lens = (270, 129, 1, 0)
    for b, n in enumerate(lens):
        for x in (q, k, v, dout):
            x[b, :, n:] = NAN
    for window, sinks in (((-1, 0), 0), ((50, 0), 3), ((20, 20), 0), ((-1, -1), 0)):
        check(q, k, v, dout, window=window, sinks=sinks, lengths=ints(*lens), starts=0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_positions_before_and_behind_the_sequence(dtype):
    q, k, v, dout = make(6, dtype, 3, 2, 2, 64, 200, 200)
    check(q, k, v, dout, window=(30, 0), starts=ints(-50, 150, 2 ** 31 - 1))
    check(q, k, v, dout, window=(30, 30), starts=ints(-2 ** 31, -199, 199), lengths=ints(1, 9, 900))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_in_front_with_garbage(dtype):
    """Sequences aligned to the right: rows before position 0 hold anything."""
    B, N = 3, 150
    q, k, v, dout = make(14, dtype, B, 4, 2, 64, N, N)
    front = (0, 45, 149)
    for b, n in enumerate(front):
        q[b, :, :n], dout[b, :, :n] = NAN, NAN
        k[b, :, N - n:], v[b, :, N - n:] = NAN, NAN
    lengths = ints(*(N - n for n in front))
    for window, sinks in (((-1, 0), 0), ((20, 0), 3), ((9, 9), 0)):
        check(q, k, v, dout, window=window, sinks=sinks, lengths=lengths)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_inputs_and_outputs(dtype):
    """Slices of a fused projection and of a longer cache, read and written in place."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    B, N, H, d = 2, 140, 3, 64
    qkv = torch.randn((B, N, 3, H, d), generator=g, device="cuda").to(DT[dtype])
    q, k, v = qkv.unbind(2)
    dout = torch.randn((B, N, H, d), generator=g, device="cuda").to(DT[dtype])
    check(q, k, v, dout, layout="bnhd", window=(33, 0))
    cache = torch.randn((2, B, H, 512, d), generator=g, device="cuda").to(DT[dtype])
    kc, vc = cache[0, :, :, 100:300], cache[1, :, :, 100:300]
    check(q.transpose(1, 2), kc, vc, window=(-1, 0))
    wide = torch.full((B, N, H, 2 * d), 7.0, device="cuda", dtype=DT[dtype])
    window_attention(q, k, v, layout="bnhd", out=wide[..., :d])
    assert torch.equal(wide[..., :d], window_attention(q, k, v, layout="bnhd"))
    assert (wide[..., d:] == 7).all()


def test_paths():
    q, k, v, _ = make(0, "bf16", 1, 4, 2, 128, 33, 64)
    assert window_attention_path(q, k, v) == 1
    assert window_attention_path(q[:, :, :32], k, v) == 2
    q, k, v, _ = make(0, "f32", 1, 4, 2, 128, 33, 64)
    assert window_attention_path(q, k, v) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq", [1, 200])
def test_large_logits(dtype, Nq):
    """One key dominates by far, and logits of +-1e4 stay finite."""
    q, k, v, dout = make(8, dtype, 1, 2, 2, 64, Nq, 200)
    q, k = q * 30, k * 30
    out, lse = window_attention(q, k, v, window=(-1, -1), return_lse=True)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    ref = attention(q, k, v, window=(-1, -1))
    assert_within(lse, ref["lse"], ref["lse_bound"], "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Nq", [1, 260])
def test_repeats_exactly_and_on_another_stream(dtype, Nq):
    q, k, v, dout = make(9, dtype, 2, 4, 2, 128, Nq, 600)
    a = window_attention(q, k, v, window=(300, 0), return_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = window_attention(q, k, v, window=(300, 0), return_lse=True)
        gb = window_attention_backward(q, k, v, *b, dout, window=(300, 0))
    s.synchronize()
    ga = window_attention_backward(q, k, v, *a, dout, window=(300, 0))
    for x, y in zip(a + ga, b + gb):
        assert torch.equal(x, y)


def test_captured_and_replayed():
    """A forward, a token call and a backward in one graph, replayed on new inputs."""
    q, k, v, dout = make(10, "bf16", 1, 4, 2, 64, 300, 300)
    q1 = q[:, :, :1].contiguous()

    def step():
        out, lse = window_attention(q, k, v, window=(99, 0), sinks=2, return_lse=True)
        return (out, lse, window_attention(q1, k, v, window=(99, 0), sinks=2),
                *window_attention_backward(q, k, v, out, lse, dout, window=(99, 0), sinks=2))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for x in (q, k, v, dout):
        x.copy_(torch.randn_like(x))
    q1.copy_(q[:, :, :1])
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(captured, step()):
        assert torch.equal(x, y)


# ---------------------------------------------------------------- how the work is divided
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64)])
@pytest.mark.parametrize("mask", [((-1, -1), 0, 1), ((-1, 0), 0, 1), ((1500, 0), 40, 1),
                                  ((2, 0), 1, 400)])
def test_few_queries_against_long_caches(dtype, d, mask):
    """Fewer query tiles than SMs against thousands of keys: the CTAs divide the line of all
    key chunks and cut problems; ragged lengths, one sequence empty, one shorter than its
    queries."""
    window, sinks, frame = mask
    lens = (6000, 0, 4097, 350)
    q, k, v, _ = make(20, dtype, 4, 3, 1, d, 600, 6000)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = NAN, NAN
    out, lse = check(q, k, v, window=window, sinks=sinks, frame=frame, lengths=ints(*lens))
    assert (out[1] == 0).all() and (out[3, :, :250] == 0).all()
    assert (lse[3, :, :250] == -float("inf")).all()
    check(q, k, v, window=window, sinks=sinks, frame=frame, lengths=ints(0, 0, 0, 0))
    check(q[:1, :1], k[:1], v[:1], window=window, sinks=sinks, frame=frame)


@pytest.mark.parametrize("B,H,Nq,Nk", [(6, 3, 1500, 5000), (33, 1, 250, 6000)])
def test_line_of_many_entries(B, H, Nq, Nk):
    """More than 32 pairs of query tiles on the line of all chunks, each with another number
    of keys: the CTAs divide it by the sums that the lanes of one warp have left to each
    other."""
    lens = [Nk - (Nk * b) // B - b % 3 for b in range(B)]
    q, k, v, _ = make(27, "bf16", B, H, 1, 64, Nq, Nk)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = NAN, NAN
    for window in ((-1, -1), (-1, 0)):
        out, lse = check(q, k, v, window=window, lengths=ints(*lens))
        for _ in range(3):
            again = window_attention(q, k, v, window=window, lengths=ints(*lens), return_lse=True)
            assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hkv,d,lens", [(2, 2, 1, 64, (40000, 3)), (1, 5, 1, 128, (30011,)),
                                            (9, 8, 8, 128, (4097, 1, 0, 65, 640, 2049, 7, 4000, 64)),
                                            (40, 2, 2, 32, None), (300, 2, 2, 64, None)])
def test_parts_of_every_number(dtype, B, H, Hkv, d, lens):
    """From one part a sequence to hundreds in many clusters, most of them empty for short
    sequences; windows that leave some parts nothing."""
    lens = list(lens or [(53 * b) % 400 for b in range(B)])
    q, k, v, _ = make(24, dtype, B, H, Hkv, d, 1, max(max(lens), 1))
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = NAN, NAN
    for window, sinks in (((-1, 0), 0), ((2999, 0), 70)):
        check(q, k, v, window=window, sinks=sinks, lengths=ints(*lens))


@pytest.mark.parametrize("d", [64, 128])
def test_more_problems_than_sms(d):
    q, k, v, dout = make(21, "bf16", 3, 64, 64, d, 300, 300)
    check(q, k, v, dout, window=(90, 0), sinks=2, lengths=ints(300, 141, 0), starts=0)


@pytest.mark.parametrize("B,H,N,lens", [(3, 64, 900, (0, 900, 300)), (2, 40, 1300, (1300, 1)),
                                        (300, 1, 300, None), (5, 3, 200, (0, 7, 200, 0, 129)),
                                        (2, 96, 300, (0, 0))])
def test_ragged_batches_over_the_ctas(B, H, N, lens):
    """Problems without keys lie among the others, over one to several rounds of CTAs."""
    q, k, v, _ = make(23, "bf16", B, H, 1, 32, N, N)
    lens = ints(*(lens or [(97 * b) % (N + 1) for b in range(B)]))
    for b, n in enumerate(lens.tolist()):
        q[b, :, n:], k[b, :, n:], v[b, :, n:] = NAN, NAN, NAN
    out, lse = check(q, k, v, window=(200, 0), sinks=1, lengths=lens, starts=0)
    for b, n in enumerate(lens.tolist()):
        assert (out[b, :, n:] == 0).all() and (lse[b, :, n:] == -float("inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (16, 1)])
def test_few_key_tiles_with_many_query_blocks(dtype, H, Hkv):
    """The query blocks of a key tile are split over CTAs (bfloat16) and joined."""
    q, k, v, dout = make(22, dtype, 1, H, Hkv, 64, 1000, 1000)
    check(q, k, v, dout, window=(-1, 0), starts=0)
    check(q, k, v, dout, window=(100, 30), sinks=3, starts=0, lengths=ints(777))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Nq,Nk", [(64, 100, 3000), (128, 70, 1500), (32, 9, 2500)])
def test_few_queries_over_many_keys_with_gradients(dtype, d, Nq, Nk):
    """Each tile's walk over the other side is divided over CTAs (float32: both passes)."""
    q, k, v, dout = make(25, dtype, 3, 6, 3, d, Nq, Nk)
    for window, sinks in (((-1, 0), 0), ((-1, -1), 0), ((900, 0), 130)):
        check(q, k, v, dout, window=window, sinks=sinks, lengths=ints(Nk, Nk // 3, 0))


@pytest.mark.parametrize("N", [64, 128, 192, 256, 320, 384, 448, 512])
def test_rows_of_few_keys_get_exact_deltas(N):
    """Around the number of key blocks up to which delta comes from the products."""
    q, k, v, dout = make(N, "bf16", 1, 2, 2, 128, N, N)
    check(q, k, v, dout, window=(-1, 0))
    check(q, k, v, dout, window=(-1, -1))


def test_heads_past_32_bit_offsets():
    """A cache whose last head starts past 2^31 elements."""
    cap, Hkv, d = 1 << 21, 9, 128
    cache = torch.empty((2, 1, Hkv, cap, d), dtype=torch.bfloat16, device="cuda")
    q, k, v, _ = make(23, "bf16", 1, Hkv, Hkv, d, 130, 200)
    cache[0, :, :, :200], cache[1, :, :, :200] = k, v
    ref = attention(q, k, v)
    for n in (130, 3):
        out = window_attention(q[:, :, 130 - n:], cache[0], cache[1], lengths=ints(200))
        assert_within(out, ref["out"][:, :, 130 - n:], ref["out_bound"][:, :, 130 - n:], "out")


def test_workspaces():
    """The caller's where it is large enough; never one that counts bytes it has not."""
    q, k, v, dout = make(15, "bf16", 1, 2, 2, 64, 90, 90)
    out, lse = window_attention(q, k, v, return_lse=True)
    mine = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    want = window_attention_backward(q, k, v, out, lse, dout)
    for ws in (mine, mine[:16], mine.view(torch.float32)):
        got = window_attention_backward(q, k, v, out, lse, dout, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for ws in (mine[:1].expand(1 << 20), mine[::2], mine.cpu()):
        with pytest.raises(ValueError):
            window_attention_backward(q, k, v, out, lse, dout, workspace=ws)


def test_wrong_arguments_are_refused():
    q, k, v, dout = make(16, "bf16", 2, 4, 2, 64, 40, 40)
    out, lse = window_attention(q, k, v, return_lse=True)
    lens = ints(40, 40)
    for bad in (dict(window=(1,)), dict(window=(1, 2, 3)), dict(window=(2 ** 40, 0)),
                dict(window=(1.5, 0)), dict(sinks=2 ** 31), dict(frame="x"), dict(scale="x"),
                dict(layout="nbhd"), dict(lengths=lens.long()), dict(lengths=lens[:1]),
                dict(lengths=lens.cpu()), dict(starts=-2 ** 31), dict(starts=2 ** 31),
                dict(starts=ints(1, 2, 3)), dict(out=q), dict(out=v), dict(out=out[:, :2]),
                dict(out=out.float()), dict(out=out.cpu())):
        with pytest.raises(ValueError):
            window_attention(q, k, v, **bad)
    for a, b, c in ((q[0], k, v), (q, k, v[:, :1]), (q, k[:1], v[:1]), (q, k.float(), v),
                    (q, k[..., :32], v[..., :32]), (q.transpose(2, 3), k, v), (q.cpu(), k, v),
                    (q, k.cpu(), v.cpu()), (q.half(), k.half(), v.half())):
        with pytest.raises(ValueError):
            window_attention(a, b, c)
    with pytest.raises(TypeError):
        window_attention(q, k, None)
    for bad in (dict(window=(-2, 0)), dict(frame=0), dict(sinks=-1), dict(scale=0.0),
                dict(scale=float("inf"))):
        with pytest.raises(_lib.MonarchError):
            window_attention(q, k, v, **bad)
    with pytest.raises(_lib.MonarchError):     # broadcast keys have no strides of their own
        window_attention(q, k[:, :1].expand(2, 2, 40, 64), v)
    for x in (lse.double(), lse[:, :, :39], lse.transpose(1, 2)):
        with pytest.raises(ValueError):
            window_attention_backward(q, k, v, out, x, dout)
    with pytest.raises(ValueError):
        window_attention_backward(q, k, v, out, lse, dout.float())
    with pytest.raises(ValueError):            # the gradient of a plain sum
        window_attention_backward(q, k, v, out, lse, torch.ones_like(q[:1, :1, :1, :1]).expand_as(q))


def test_paged_wrong_arguments_are_refused():
    q = torch.randn(2, 4, 64, device="cuda")
    pool = torch.randn(6, 2, 16, 64, device="cuda")
    table, lens = ints(0, 1, 2, 3, 4, 5).view(2, 3), ints(20, 48)
    paged_attention(q, pool, pool, table, lens)
    for args in ((q[0], pool, pool, table, lens), (q, pool, pool[:3], table, lens),
                 (q, pool[..., :32], pool[..., :32], table, lens), (q, pool, pool, table[0], lens),
                 (q, pool, pool, table.long(), lens), (q, pool, pool, table[:, :0], lens),
                 (q, pool, pool, table[:1], lens), (q, pool, pool, table, lens.long()),
                 (q, pool, pool, table.cpu(), lens), (q, pool.bfloat16(), pool.bfloat16(), table, lens)):
        with pytest.raises(ValueError):
            paged_attention(*args)
    with pytest.raises(ValueError):
        paged_attention(q, pool, pool, table, lens, out=q)
    with pytest.raises(TypeError):
        paged_attention(q, pool, pool, table, None)
    with pytest.raises(_lib.MonarchError):     # pages of 12
        paged_attention(q, pool[:, :, :12], pool[:, :, :12], table, lens)


def test_waits_give_up_and_the_next_call_is_right():
    """Fault injection on the host: the issuing threads wait on a barrier that nothing
    completes, give up after a short limit, and the status says so."""
    q, k, v, dout = make(24, "bf16", 1, 2, 2, 128, 300, 300)
    out, lse = window_attention(q, k, v, return_lse=True)
    torch.cuda.synchronize()
    old = _lib.monarch_set_wait_limit(2000)
    _lib.monarch_debug_inject_stall(True)
    try:
        window_attention(q, k, v)
        assert _lib.monarch_last_device_status(None) == 7   # MONARCH_ERR_TIMEOUT
        window_attention_backward(q, k, v, out, lse, dout)
        assert _lib.monarch_last_device_status(None) == 7
    finally:
        _lib.monarch_debug_inject_stall(False)
        _lib.monarch_set_wait_limit(old)
    check(q, k, v, dout)


def test_wait_limit_is_not_a_limit_on_the_length():
    """A CTA's epilogue waits for all of a problem's blocks (here 3125, for 2 ms).  With a limit
    on polls that this wait passes, and each block's own waits do not, the call completes."""
    H = torch.cuda.get_device_properties(0).multi_processor_count
    q, k, v, _ = make(28, "bf16", 1, H, 1, 64, 256, 200000)
    want = window_attention(q, k, v, window=(-1, -1))
    torch.cuda.synchronize()
    old = _lib.monarch_set_wait_limit(256)
    try:
        got = window_attention(q, k, v, window=(-1, -1))
        assert _lib.monarch_last_device_status(None) == 0
    finally:
        _lib.monarch_set_wait_limit(old)
    assert torch.equal(got, want)


# ---------------------------------------------------------------- paged
def pages_of(k, v, page, lengths, layout, seed=0, extra=3):
    """Scattered pages that hold each sequence's keys, and NaN everywhere else."""
    B, Hkv, Nk, d = k.shape
    width = -(-Nk // page)
    need = [-(-n // page) for n in lengths]
    total = sum(need) + extra
    g = torch.Generator()
    g.manual_seed(seed)
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((B, width), -1, dtype=torch.int32)
    kp, vp = (torch.full((total, Hkv, page, d), NAN, device="cuda", dtype=k.dtype)
              for _ in range(2))
    at = 0
    for b, n in enumerate(lengths):
        for i in range(need[b]):
            pg = order[at]
            at += 1
            table[b, i] = pg
            m = min(page, n - i * page)
            kp[pg, :, :m] = k[b, :, i * page:i * page + m]
            vp[pg, :, :m] = v[b, :, i * page:i * page + m]
    if layout == "bnhd":
        kp, vp = kp.transpose(1, 2).contiguous(), vp.transpose(1, 2).contiguous()
    return kp, vp, table.cuda()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 128)])
@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 1), (20, 1)])
def test_paged(dtype, d, page, H, Hkv):
    lengths = (1, 7, 500, 0, 1201)
    q, k, v, _ = make(11, dtype, 5, H, Hkv, d, 1, 1201)
    for layout in ("bhnd", "bnhd"):
        kp, vp, table = pages_of(k, v, page, lengths, layout)
        for window, sinks in (((-1, 0), 0), ((200, 0), 3), ((0, 0), 0)):
            mask = dict(window=window, sinks=sinks)
            ref = attention(q, k, v, lengths=ints(*lengths), **mask)
            out, lse = paged_attention(q[:, :, 0], kp, vp, table, ints(*lengths), layout=layout,
                                       return_lse=True, **mask)
            assert_within(out, ref["out"][:, :, 0], ref["out_bound"][:, :, 0], "out")
            assert_within(lse, ref["lse"], ref["lse_bound"], "lse")
            assert (out[3] == 0).all()
    _lib.check(_lib.monarch_last_device_status(None), "device status")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_with_pages_given_back(dtype):
    """Behind the sinks and before the window the table holds no pages."""
    n, page = 1000, 8
    q, k, v, _ = make(12, dtype, 1, 4, 2, 64, 1, n)
    kp, vp, table = pages_of(k, v, page, (n,), "bhnd")
    ref = attention(q, k, v, window=(99, 0), sinks=3)
    table[0, 1:(n - 100) // page] = -1
    out = paged_attention(q[:, :, 0], kp, vp, table, ints(n), window=(99, 0), sinks=3)
    assert_within(out, ref["out"][:, :, 0], ref["out_bound"][:, :, 0], "out")
    torch.cuda.synchronize()
    _lib.check(_lib.monarch_last_device_status(None), "device status")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_page_is_reported_and_its_keys_absent(dtype):
    n, page = 96, 16
    q, k, v, _ = make(13, dtype, 1, 2, 2, 64, 1, n)
    kp, vp, table = pages_of(k, v, page, (n,), "bhnd")
    rest = torch.cat([torch.arange(32), torch.arange(48, n)]).cuda()
    ref = attention(q, k[:, :, rest], v[:, :, rest])
    for bad in (-1, kp.shape[0], 2 ** 31 - 1):
        table[0, 2] = bad
        out = paged_attention(q[:, :, 0], kp, vp, table, ints(n))
        assert _lib.monarch_last_device_status(None) == 1   # MONARCH_ERR_INVALID_ARG
        assert_within(out, ref["out"][:, :, 0], ref["out_bound"][:, :, 0], "out")
    assert _lib.monarch_last_device_status(None) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_paged_long_cache(dtype):
    lengths = (40000, 12345)
    q, k, v, _ = make(14, dtype, 2, 8, 1, 128, 1, 40000)
    kp, vp, table = pages_of(k, v, 64, lengths, "bhnd")
    ref = attention(q, k, v, lengths=ints(*lengths))
    out = paged_attention(q[:, :, 0], kp, vp, table, ints(*lengths))
    assert_within(out, ref["out"][:, :, 0], ref["out_bound"][:, :, 0], "out")


def test_paged_pool_past_32_bit_offsets():
    """Pages whose elements lie past 2^31: 70,000 pages of 64 x 4 x 128."""
    pages, page, Hkv, d = 70000, 64, 4, 128
    pool = torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    q, k, v, _ = make(15, "bf16", 1, 8, Hkv, d, 1, 128)
    at = [pages - 1, pages - 3]
    vpool = torch.empty_like(pool)
    for i, pg in enumerate(at):
        pool[pg] = k[0, :, i * page:(i + 1) * page]
        vpool[pg] = v[0, :, i * page:(i + 1) * page]
    ref = attention(q, k, v)
    out = paged_attention(q[:, :, 0], pool, vpool, ints(*at).view(1, 2), ints(128))
    assert_within(out, ref["out"][:, :, 0], ref["out_bound"][:, :, 0], "out")
