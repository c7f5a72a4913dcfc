"""Window, paged and rotary entry points without a GPU: what they refuse, before
anything is enqueued, and the rotary frequencies."""
import glob
import math
import os
import re

import pytest
import torch

from structured_attention_video_b200 import _lib, rotary, rotary_frequencies, window_attention

P = 1 << 20   # never dereferenced: validation fails first
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, NO_MEMORY = range(6)


def desc(**kw):
    d = _lib.WindowDesc()
    d.B, d.H, d.Hkv, d.Nq, d.Nk, d.d = 2, 8, 2, 100, 200, 64
    d.frame, d.left, d.right, d.sinks, d.start = 1, 10, 0, 1, 0
    d.dtype, d.scale = _lib.BF16, 0.125
    for s in (d.q, d.k, d.v, d.out):
        s.batch, s.head, s.token = 8 * 200 * 64, 200 * 64, 64
    for name, x in kw.items():
        if "." in name:
            a, b = name.split(".")
            setattr(getattr(d, a), b, x)
        else:
            setattr(d, name, x)
    return d


def fwd(d, q=P, k=P, v=P, out=P, lse=None, ws=P, n=1 << 40):
    return _lib.monarch_window_attn_fwd_ws(d, q, k, v, out, lse, ws, n, None)


BAD = [({"B": 0}, INVALID), ({"Nq": 0}, INVALID), ({"Nk": -1}, INVALID), ({"frame": 0}, INVALID),
       ({"left": -2}, INVALID), ({"right": -2}, INVALID), ({"sinks": -1}, INVALID),
       ({"dtype": 2}, INVALID), ({"scale": 0.0}, INVALID), ({"scale": -1.0}, INVALID),
       ({"scale": math.inf}, INVALID), ({"scale": math.nan}, INVALID), ({"d": 96}, UNSUPPORTED),
       ({"d": 256}, UNSUPPORTED), ({"Hkv": 3}, SHAPE), ({"B": 9000}, SHAPE),
       ({"Nk": 2 ** 30 + 1}, SHAPE), ({"q.token": 0}, INVALID), ({"k.head": -64}, INVALID),
       ({"v.token": 65}, ALIGN), ({"out.head": 4}, ALIGN), ({"k.batch": 1 << 40}, SHAPE)]


@pytest.mark.parametrize("kw,code", BAD)
def test_window_refusals(kw, code):
    d = desc(**kw)
    assert fwd(d) == code
    assert _lib.monarch_window_attn_workspace_bytes(d) == 0
    assert _lib.monarch_window_attn_bwd_workspace_bytes(d) == 0
    assert _lib.monarch_window_attn_path(d) == -1
    g = _lib.WindowGrads()
    assert _lib.monarch_window_attn_bwd_ws(d, g, *[P] * 10, 1 << 40, None) == code
    d.Nq = min(d.Nq, 1)
    d.lengths = P
    assert _lib.monarch_paged_attn_ws(d, P, P, P, P, 25, 8, 9, P, None, P, 1 << 40, None) == code


def test_window_pointers_and_workspace():
    d = desc()
    for i in range(4):
        x = [P] * 4
        x[i] = None
        assert fwd(d, *x) == INVALID
        x[i] = P + 8
        assert fwd(d, *x) == ALIGN
    assert fwd(d, lse=P + 2) == ALIGN and fwd(desc(lengths=P + 1)) == ALIGN
    assert _lib.monarch_window_attn_workspace_bytes(d) == 256   # none needed
    token = desc(Nq=1, Nk=100000, left=-1)
    need = _lib.monarch_window_attn_workspace_bytes(token)
    assert need > 256 and fwd(token, n=need - 1) == NO_MEMORY
    assert fwd(token, ws=None) == INVALID and fwd(token, ws=P + 16) == ALIGN
    assert fwd(None) == INVALID
    g = _lib.WindowGrads()
    back = lambda *x: _lib.monarch_window_attn_bwd_ws(d, *x, 1 << 40, None)   # noqa: E731
    assert back(g, *[P] * 10) == INVALID                       # no strides
    for s in (g.dout, g.dq, g.dk, g.dv):
        s.batch, s.head, s.token = 8 * 200 * 64, 200 * 64, 64
    for i in range(10):
        x = [P] * 10
        x[i] = None
        assert back(g, *x) == INVALID
    assert back(None, *[P] * 10) == INVALID
    assert _lib.monarch_window_attn_bwd_ws(d, g, *[P] * 10, 2 * 8 * 100 * 4 - 1, None) == NO_MEMORY


def test_paths():
    assert _lib.monarch_window_attn_path(desc(Nq=16)) == 2
    assert _lib.monarch_window_attn_path(desc(Nq=17)) == 1
    assert _lib.monarch_window_attn_path(desc(Nq=17, dtype=_lib.F32)) == 0


def test_paged_refusals():
    d = desc(Nq=1, Nk=200, lengths=P)
    call = lambda d=d, table=P, stride=25, page=8, pages=9: _lib.monarch_paged_attn_ws(  # noqa: E731
        d, P, P, P, table, stride, page, pages, P, None, P, 1 << 40, None)
    assert call(table=None) == INVALID and call(table=P + 2) == ALIGN
    assert call(pages=0) == INVALID
    for page in (0, 4, 12, 131072, -8):
        assert call(page=page) == UNSUPPORTED
    assert call(stride=24) == SHAPE and call(page=16) == SHAPE      # 200 is not 16 * n
    assert call(d=desc(Nq=2, lengths=P)) == SHAPE
    assert call(d=desc(Nq=1)) == INVALID                             # no lengths
    assert _lib.monarch_paged_attn_workspace_bytes(desc(Nq=2)) == 0


def rotary_desc(**kw):
    d = _lib.RotaryDesc()
    d.B, d.N, d.H, d.Hkv, d.d, d.pairs, d.axes = 2, 30, 4, 2, 64, 32, 1
    d.pairs_of_axis[0] = 32
    d.dtype, d.magnitude = _lib.BF16, 1.0
    for s in (d.q, d.k, d.q_out, d.k_out):
        s.batch, s.head, s.token = 4 * 30 * 64, 30 * 64, 64
    for name, x in kw.items():
        if name == "split":
            d.axes = len(x)
            d.pairs_of_axis[:] = list(x) + [0] * (3 - len(x))
        elif "." in name:
            a, b = name.split(".")
            setattr(getattr(d, a), b, x)
        else:
            setattr(d, name, x)
    return d


@pytest.mark.parametrize("kw,code", [
    ({"B": 0}, INVALID), ({"N": 0}, INVALID), ({"H": 0}, INVALID), ({"Hkv": -1}, INVALID),
    ({"pairs": 0}, INVALID), ({"axes": 0}, INVALID), ({"axes": 4}, INVALID), ({"half": 2}, INVALID),
    ({"inverse": -1}, INVALID), ({"dtype": 9}, INVALID), ({"magnitude": math.nan}, INVALID),
    ({"Hkv": 0}, INVALID), ({"d": 60}, UNSUPPORTED), ({"d": 2048}, UNSUPPORTED),
    ({"pairs": 33}, SHAPE), ({"split": (16, 8)}, SHAPE), ({"split": (16, 8, 8)}, INVALID),
    ({"split": (32, -8, 8)}, INVALID), ({"grid_h": 3, "grid_w": 10}, INVALID),
    ({"positions": P, "start": 1}, INVALID), ({"positions": P, "pos_token": -1}, INVALID),
    ({"positions": P + 1}, ALIGN), ({"starts": P + 2}, ALIGN), ({"q.token": 0}, INVALID),
    ({"k_out.head": 4}, ALIGN),
])
def test_rotary_refusals(kw, code):
    assert _lib.monarch_rotary(rotary_desc(**kw), P, P, P, P, P, None) == code


def test_rotary_pointers():
    d = rotary_desc()
    for i in range(5):
        x = [P] * 5
        x[i] = None
        assert _lib.monarch_rotary(d, *x, None) == INVALID
        x[i] = P + 4
        assert _lib.monarch_rotary(d, *x, None) == ALIGN
    assert _lib.monarch_rotary(None, P, P, P, P, P, None) == INVALID


def test_rotary_outputs_in_the_place_of_others_are_refused():
    d, A, B_, C = rotary_desc(), P, 2 * P, 3 * P
    call = lambda d, q, k, qo, ko: _lib.monarch_rotary(d, q, k, P, qo, ko, None)   # noqa: E731
    assert call(d, A, B_, B_, A) == INVALID      # swapped
    assert call(d, A, B_, C, C) == INVALID       # both in one place
    assert call(d, A, A, A, C) == INVALID        # queries in place that are the keys as well
    assert call(d, A, B_, C, A) == INVALID
    for name, i in (("q_out", 0), ("k_out", 1)):   # in place, tokens and heads exchanged
        x = rotary_desc(**{name + ".head": 64, name + ".token": 4 * 64})
        outs = [C, 4 * P]
        outs[i] = (A, B_)[i]
        assert call(x, A, B_, *outs) == INVALID


def test_rotary_frequencies():
    f, m = rotary_frequencies(64, device="cpu")
    want = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], dtype=torch.float64)
    assert torch.allclose(f, want, rtol=1e-14) and m == 1.0
    g, m = rotary_frequencies((8, 6, 0), base=500.0, scaling="linear", factor=4, device="cpu")
    want = torch.tensor([500.0 ** (-i / 4) / 4 for i in range(4)] +
                        [500.0 ** (-i / 3) / 4 for i in range(3)], dtype=torch.float64)
    assert torch.allclose(g, want, rtol=1e-14)
    n, _ = rotary_frequencies(64, scaling="ntk", factor=8, device="cpu")
    assert n[0] == 1.0 and math.isclose(n[-1], f[-1] / 8, rel_tol=1e-12)
    y, m = rotary_frequencies(128, scaling="yarn", factor=16, original=4096, device="cpu")
    f, _ = rotary_frequencies(128, device="cpu")
    assert math.isclose(m, 0.1 * math.log(16) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(y[turns > 40], f[turns > 40])
    assert torch.allclose(y[turns < 0.8], f[turns < 0.8] / 16, rtol=1e-14)
    ratio = f / y
    assert (ratio[1:] >= ratio[:-1] - 1e-12).all() and ratio.max() <= 16 + 1e-9


@pytest.mark.parametrize("kw", [
    dict(base=1.0), dict(scaling="linear", factor=0.5), dict(scaling="yarn", factor=2.0),
    dict(scaling="yarn", factor=2.0, original=100, beta_fast=1.0), dict(base=math.inf)])
def test_rotary_frequency_refusals(kw):
    with pytest.raises(_lib.MonarchError):
        rotary_frequencies(64, device="cpu", **kw)
    with pytest.raises(ValueError):
        rotary_frequencies(63, device="cpu")
    with pytest.raises(ValueError):
        rotary_frequencies(64, scaling="other", device="cpu")


def test_cpu_tensors_are_refused():
    q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError):
        window_attention(q, q, q)
    with pytest.raises(ValueError):
        rotary(q, q, torch.ones(32, dtype=torch.float64))


def test_wait_limit_stays_below_what_kernels_multiply():
    """16 times and more of a limit near 2^63 would be negative: every wait would give up."""
    old = _lib.monarch_set_wait_limit(2 ** 63 - 1)
    try:
        assert _lib.monarch_set_wait_limit(12345) == 2 ** 40
        assert _lib.monarch_set_wait_limit(0) == 12345
    finally:
        _lib.monarch_set_wait_limit(old)


def functions(source):
    """(name, body) of the functions of a C++ file whose braces open at namespace level."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", source, flags=re.S)
    depth, at, spaces = 0, 0, []
    for m in re.finditer(r"[{}]", text):
        if m.group() == "{":
            head = text[at:m.start()]
            spaces.append((re.search(r"\bnamespace\b[^;]*$", head) is not None, head, m.end()))
        else:
            namespace, head, begin = spaces.pop()
            if not namespace and all(n for n, _, _ in spaces):
                names = re.findall(r"(\w+)\s*\(", re.split(r"[;}]", head)[-1])
                yield (names[-1] if names else ""), text[begin:m.start()]
        at = m.end()


def test_a_cta_reads_its_sequence_once():
    """Trip counts and barriers of a CTA follow from lengths[b] and starts[b].  They are read
    in one function, and by every thread for itself only where no barrier depends on them."""
    csrc = os.path.join(os.path.dirname(_lib.__file__), "csrc")
    reads, calls, per_cta = set(), set(), set()
    for path in glob.glob(os.path.join(csrc, "window_*.cu*")):
        for name, body in functions(open(path).read()):
            if re.search(r"\b(lengths|starts)\s*\[", body):
                reads.add(name)
            if re.search(r"\bsequence\(", body):
                calls.add(name)
            if "share_sequence(" in body:
                per_cta.add(name)
    assert reads == {"sequence"}
    # one thread for all, or into the CTA's list; a row's sum or store of its own
    assert calls == {"first_threads_sequence", "token_bf16_kernel", "list_segments",
                     "row_delta_kernel"}
    assert per_cta == {"token_f32_kernel", "simt_fwd_kernel", "simt_dq_kernel", "simt_dkv_kernel",
                       "mma_dq_kernel", "mma_dkv_kernel"}
