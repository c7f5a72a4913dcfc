"""Rotary positions against complex rotation in 64 bits, and their backward."""
import pytest
import torch

from structured_attention_video_b200 import _lib, rotary, rotary_backward, rotary_frequencies

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def reference(x, pos, freqs, style, layout, magnitude=1.0, inverse=False):
    """pos [B or 1, N, pairs] (the position of each pair's axis)."""
    pairs = freqs.numel()
    t = pos.double() * freqs
    unit = torch.polar(torch.full_like(t, magnitude), -t if inverse else t)
    unit = unit[:, None] if layout == "bhnd" else unit[:, :, None]
    y = x.double()
    part, rest = y[..., :2 * pairs], y[..., 2 * pairs:]
    if style == "interleaved":
        z = torch.view_as_complex(part.unflatten(-1, (pairs, 2)).contiguous()) * unit
        part = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(part[..., :pairs], part[..., pairs:]) * unit
        part = torch.cat((z.real, z.imag), -1)
    return torch.cat((part, rest), -1)


def check(got, want, x, dtype, magnitude=1.0):
    """One rounding to the type, and sin, cos and the two products in float32: each
    within 2^-22 of the pair's length (sincospi to 2 ulp, its argument to 2^-24 of an
    eighth of a turn)."""
    length = x.double().abs().amax() * 2 ** 0.5 * abs(magnitude)
    bound = U[dtype] * want.abs() + 2.0 ** -21 * length
    err = (got.double() - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


def make(seed, dtype, B, H, N, d, layout):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = (B, H, N, d) if layout == "bhnd" else (B, N, H, d)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["interleaved", "half"])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("d,width", [(128, 128), (64, 32), (128, 20), (32, 2), (80, 72), (256, 256)])
def test_one_axis(dtype, style, layout, d, width):
    freqs, _ = rotary_frequencies(width)
    B, N = 2, 37
    q, k = make(1, dtype, B, 4, N, d, layout), make(2, dtype, B, 2, N, d, layout)
    for start in (0, 1000003, -5):
        pos = (start + torch.arange(N, device="cuda"))[None, :, None].expand(1, N, width // 2)
        for fn, inverse in ((rotary, False), (rotary_backward, True)):
            a, b = fn(q, k, freqs, style=style, layout=layout, start=start)
            check(a, reference(q, pos, freqs, style, layout, inverse=inverse), q, dtype)
            check(b, reference(k, pos, freqs, style, layout, inverse=inverse), k, dtype)
            assert torch.equal(a[..., width:], q[..., width:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["interleaved", "half"])
def test_three_axes_on_a_grid(dtype, style):
    grid, dims, d = (3, 5, 7), (44, 42, 42), 128
    N = 105
    freqs, _ = rotary_frequencies(dims)
    q, k = make(3, dtype, 2, 3, N, d, "bnhd"), make(4, dtype, 2, 3, N, d, "bnhd")
    n = torch.arange(N, device="cuda")
    axis = torch.tensor([0] * 22 + [1] * 21 + [2] * 21, device="cuda")
    first = torch.tensor([4, 90001], dtype=torch.int32, device="cuda")
    at = torch.stack([torch.stack((f + n // 35, n // 7 % 5, n % 7), -1) for f in first.long()])
    a, b = rotary(q, k, freqs, dims=dims, style=style, grid=grid, start=first, layout="bnhd")
    check(a, reference(q, at[..., axis], freqs, style, "bnhd"), q, dtype)
    check(b, reference(k, at[..., axis], freqs, style, "bnhd"), k, dtype)
    # the same positions given as a tensor
    c, e = rotary(q, k, freqs, dims=dims, style=style, positions=at.int(), layout="bnhd")
    assert torch.equal(a, c) and torch.equal(b, e)


def test_far_positions_keep_their_accuracy():
    freqs, _ = rotary_frequencies(128, base=1e6)
    q = make(5, "f32", 1, 1, 64, 128, "bhnd")
    pos = torch.randint(2 ** 30, 2 ** 31 - 1, (64,), dtype=torch.int32, device="cuda")
    a, none = rotary(q, None, freqs, positions=pos)
    assert none is None
    # the reference in 64 bits is itself off by position * 2^-53
    check(a, reference(q, pos[None, :, None], freqs, "interleaved", "bhnd"), q, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_strided_and_magnitude(dtype):
    freqs, magnitude = rotary_frequencies(32, scaling="yarn", factor=4.0, original=256)
    assert magnitude > 1.1
    B, N, H, d = 2, 50, 3, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    qkv = torch.randn((B, N, 3, H, d), generator=g, device="cuda").to(DT[dtype])
    before = qkv.clone()
    q, k, v = qkv.unbind(2)
    pos = torch.arange(N, device="cuda")[None, :, None]
    rotary(q, k, freqs, style="half", layout="bnhd", magnitude=magnitude, out=(q, k))
    for i, x in enumerate((q, k)):
        want = reference(before[:, :, i], pos, freqs, "half", "bnhd", magnitude)
        check(x, want, before[:, :, i], dtype, magnitude)
    assert torch.equal(v, before[:, :, 2])
    cache = torch.zeros((B, H, 200, d), device="cuda", dtype=DT[dtype])
    kn = before[:, :, 1].transpose(1, 2)
    qn = before[:, :, 0].transpose(1, 2)
    a, _ = rotary(qn, kn, freqs, start=70, out=(torch.empty_like(qn), cache[:, :, 70:120]))
    b, c = rotary(qn, kn, freqs, start=70)
    assert torch.equal(a, b) and torch.equal(cache[:, :, 70:120], c)
    assert (cache[:, :, :70] == 0).all() and (cache[:, :, 120:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("style", ["interleaved", "half"])
@pytest.mark.parametrize("width", [2, 6, 20])
def test_elements_that_do_not_turn_are_copied(dtype, style, width):
    """Bit for bit, whatever they hold and wherever the turned part ends."""
    freqs, _ = rotary_frequencies(width)
    q = make(10, dtype, 2, 3, 9, 32, "bhnd")
    rest = q[..., width:]
    rest[..., 0::4], rest[..., 1::4], rest[..., 2::4] = float("inf"), float("nan"), -0.0
    a, _ = rotary(q, None, freqs, style=style, start=3)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(a[..., width:].contiguous().view(bits), rest.contiguous().view(bits))
    pos = (3 + torch.arange(9, device="cuda"))[None, :, None].expand(1, 9, width // 2)
    q[..., width:] = 0
    a, _ = rotary(q, None, freqs, style=style, start=3)
    check(a, reference(q, pos, freqs, style, "bhnd"), q, dtype)


def test_wrong_arguments_are_refused():
    freqs, _ = rotary_frequencies(32)
    q, k = make(11, "f32", 2, 4, 24, 64, "bhnd"), make(12, "f32", 2, 2, 24, 64, "bhnd")
    pos = torch.arange(24, dtype=torch.int32, device="cuda")
    rotary(q, k, freqs, positions=pos[None].expand(2, 24))
    for bad in (dict(style="whole"), dict(layout="nbhd"), dict(dims=(32, 2)), dict(dims=(31, 1)),
                dict(dims=()), dict(dims=(8, 8, 8, 8)), dict(dims=(-2, 34)),
                dict(dims=(8, 12, 12), grid=(2, 3, 5)), dict(dims=(8, 12, 12), grid=(2, 12)),
                dict(positions=pos.long()), dict(positions=pos[:23]), dict(positions=pos.cpu()),
                dict(positions=pos.expand(3, 24)), dict(positions=pos, dims=(8, 12, 12)),
                dict(positions=pos[:, None].expand(24, 3), dims=(8, 12, 12)), dict(start=2 ** 31),
                dict(start=pos), dict(start=1.5), dict(magnitude="x"), dict(out=(q,)),
                dict(out=(q, None)), dict(out=(q[:1], k)), dict(out=(q, k.bfloat16()))):
        with pytest.raises(ValueError):
            rotary(q, k, freqs, **bad)
    for a, b, f in ((q[0], k, freqs), (q, k[:, :, :23], freqs), (q, k.bfloat16(), freqs),
                    (q, k, freqs.float()), (q, k, freqs.cpu()), (q, k, freqs[::2]),
                    (q.cpu(), None, freqs), (q, k.cpu(), freqs), (q.transpose(2, 3), None, freqs)):
        with pytest.raises(ValueError):
            rotary(a, b, f)
    with pytest.raises(_lib.MonarchError):      # more pairs than the head has
        rotary(q[..., :16], None, freqs)
    with pytest.raises(_lib.MonarchError):      # three axes without a grid or positions
        rotary(q, k, freqs, dims=(8, 12, 12))


def test_backward_is_the_gradient():
    """Against central differences of the forward's 64-bit form along a direction."""
    freqs, _ = rotary_frequencies((8, 12, 12))
    q, d = make(7, "f32", 1, 2, 24, 32, "bhnd"), make(8, "f32", 1, 2, 24, 32, "bhnd")
    w = make(9, "f32", 1, 2, 24, 32, "bhnd")
    kw = dict(dims=(8, 12, 12), grid=(2, 3, 4), start=9)
    dq, _ = rotary_backward(w, None, freqs, **kw)
    f = lambda x: float((rotary(x, None, freqs, **kw)[0].double() * w.double()).sum())  # noqa: E731
    slope = (f(q + d) - f(q - d)) / 2     # the map is linear: exact but for roundings
    assert abs(slope - float((dq.double() * d.double()).sum())) < 1e-3


def test_outputs_in_the_place_of_others_are_refused():
    freqs, _ = rotary_frequencies(64)
    q, k = make(13, "f32", 1, 24, 24, 64, "bhnd"), make(14, "f32", 1, 24, 24, 64, "bhnd")
    before = q.clone(), k.clone()
    new = torch.empty_like(q)
    for a, b, out in ((q, k, (k, q)), (q, k, (new, new)), (q, q, (q, new)),
                      (q, k, (q.transpose(1, 2), k))):
        with pytest.raises(_lib.MonarchError):
            rotary(a, b, freqs, out=out)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    a, b = rotary(q, k, freqs)
    c, d = rotary(q, q, freqs)      # the same queries and keys, each turned into its own place
    assert torch.equal(a, c) and torch.equal(c, d)
    rotary(q, k, freqs, out=(q, k))
    assert torch.equal(q, a) and torch.equal(k, b)
