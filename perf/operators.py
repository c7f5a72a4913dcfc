"""Measured cases of the exact-attention operators next to the Monarch attention.

Four operators, each with a plain form in elementary torch operations and the
framework's own call:

  window   softmax attention over a window of frames and the first frames (sinks),
           forward: the newest tokens against a cache, or a whole sequence
  train    the same, forward and backward
  paged    one new token a sequence over a paged key/value cache
  rotary   rotary positions of queries and keys, one axis or (frame, row, column),
           forward and backward

Masks.  Key j of sequence b exists when j < lengths[b].  Query i sits at position
p = starts[b] + i and is a real row when 0 <= p < lengths[b]; other rows give
zeros.  With fq = p // frame and fk = j // frame it sees key j when fk <= fq + right
(right >= 0) and fk >= fq - left (left >= 0) or fk < sinks.
"""
import math

import torch

own = False

_ops = None


def _framework():
    """The framework's public operators, imported at the first call that needs them."""
    global _ops
    if _ops is None:
        import structured_attention_video_b200 as _ops
    return _ops


_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _window(name, dtype, B, H, Hkv, d, Nq, Nk, frame, left, right, sinks, lengths, layout):
    return {"name": name, "op": "window", "dtype": dtype, "B": B, "H": H, "Hkv": Hkv, "d": d,
            "Nq": Nq, "Nk": Nk, "frame": frame, "left": left, "right": right, "sinks": sinks,
            "lengths": lengths, "layout": layout}


def _train(name, dtype, B, H, Hkv, d, N, frame, left, right, sinks, lengths, layout):
    c = _window(name, dtype, B, H, Hkv, d, N, N, frame, left, right, sinks, lengths, layout)
    return dict(c, op="train")


def _paged(name, dtype, B, H, Hkv, d, page, most, left, sinks):
    return {"name": name, "op": "paged", "dtype": dtype, "B": B, "H": H, "Hkv": Hkv, "d": d,
            "page": page, "most": most, "frame": 1, "left": left, "right": 0, "sinks": sinks}


def _rotary(name, dtype, B, N, H, Hkv, d, axes, style, first, factor, layout, backward):
    return {"name": name, "op": "rotary", "dtype": dtype, "B": B, "N": N, "H": H, "Hkv": Hkv,
            "d": d, "axes": axes, "style": style, "first": first, "factor": factor,
            "layout": layout, "backward": backward}


def listed():
    return [
        # a new chunk of three 480p frames (30 x 52 tokens each) in a rollout: its queries
        # see the first chunk of the clip and the last two chunks besides their own, in a
        # cache of 21 frames
        _window("window_chunk_480p", "bf16", 1, 12, 12, 128, 4680, 32760, 4680, 2, 0, 1, "full",
                "bhnd"),
        # prompts of two lengths in one padded batch, causal, the last 1024 tokens and the
        # first four, four query heads to a key head
        _window("window_prompts", "bf16", 2, 16, 4, 64, 4001, 4001, 1, 1023, 0, 4, "ragged",
                "bnhd"),
        # one new token a sequence against an ordinary (not paged) cache, everything visible
        _window("window_token", "bf16", 8, 32, 8, 128, 1, 4097, 1, -1, 0, 0, "ragged", "bhnd"),
        # the smallest clip in 32 bits: three frames of 8 x 8 tokens, each frame sees itself
        # and the one before
        _window("window_tiny_f32", "f32", 1, 2, 2, 32, 192, 192, 64, 1, 0, 0, "full", "bhnd"),
        # training on nine 480p frames, every frame sees itself, the two before and the first
        _train("train_480p", "bf16", 1, 12, 12, 128, 14040, 1560, 2, 0, 1, "full", "bhnd"),
        # causal training on a padded batch of short sequences with shared key heads
        _train("train_short_gqa", "bf16", 2, 8, 2, 64, 1023, 1, -1, 0, 0, "ragged", "bnhd"),
        # training in 32 bits, a window to both sides
        _train("train_f32", "f32", 1, 4, 4, 64, 780, 1, 127, 127, 0, "full", "bhnd"),
        # the first tokens of one sequence: latency counts
        _paged("paged_first", "bf16", 1, 12, 12, 128, 16, 333, -1, 0),
        # sixteen sequences of many lengths up to 8192
        _paged("paged_batch", "bf16", 16, 32, 8, 128, 64, 8192, -1, 0),
        # four very long caches
        _paged("paged_long", "bf16", 4, 40, 8, 128, 64, 131072, -1, 0),
        # queries and keys of a 720p clip, 21 frames of 45 x 80 tokens, the head split over
        # (frame, row, column)
        _rotary("rotary_720p", "bf16", 1, 75600, 12, 12, 128, "44,42,42", "interleaved", 0, 1.0,
                "bnhd", False),
        # the gradients of a batch's queries and keys in 32 bits, half of each head rotated,
        # positions interpolated four times
        _rotary("rotary_train", "f32", 2, 4001, 16, 4, 64, "32", "half", 100000, 4.0, "bnhd",
                True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "train", "paged", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 128])
    layout = rng.choice(["bhnd", "bnhd"])
    if op == "rotary":
        Hkv = rng.choice([1, 2, 4, 8, 12])
        H = Hkv * rng.choice([1, 2, 4])
        B = rng.choice([1, 2, 3])
        N = _log(rng, 1, max(2, 75600 * 24 // (B * (H + Hkv) * (1 if dtype == "bf16" else 2))))
        axes = rng.choice(["%d" % d, "%d" % (d // 2), "%d,%d,%d" % (d - 4 * (d // 6), 2 * (d // 6),
                                                                     2 * (d // 6))])
        c = _rotary("", dtype, B, min(N, 75600), H, Hkv, d, axes,
                    rng.choice(["interleaved", "half"]), _log(rng, 1, 1000000),
                    rng.choice([1.0, 2.0, 8.0]), layout, rng.random() < 0.4)
    elif op == "paged":
        Hkv = rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 32)
        page = rng.choice([8, 16, 32, 64, 128])
        most = _log(rng, 1, min(131072, 131072 * 32 * 128 // (2 * B * Hkv * d)))
        left = rng.choice([-1, -1, _log(rng, 1, 4096)])
        c = _paged("", dtype, B, Hkv * rng.choice([1, 2, 5, 8]), Hkv, d, page, most, left,
                   0 if left < 0 else rng.choice([0, 4, 64]))
    else:
        Hkv = rng.choice([1, 2, 3, 4])
        H = Hkv * rng.choice([1, 2, 4])
        B = rng.choice([1, 2, 3])
        # at most 6e8 pairs of a query and a key over all heads
        most = int(math.sqrt(6e8 / (B * H)))
        frame = rng.choice([1, 1, 1, 64, 390, 1560])
        reach = max(1, most // frame)
        left = rng.choice([-1, _log(rng, 1, reach)])
        right = rng.choice([0, 0, -1, _log(rng, 1, reach)])
        sinks = rng.choice([0, 1, 4]) if left >= 0 else 0
        lengths = rng.choice(["full", "ragged"])
        if op == "train":
            # from 16 tokens on: a row that sees one key has dq = 0, which leaves nothing to
            # compare with when it is the only one
            c = _train("", dtype, B, H, Hkv, d, _log(rng, 16, min(8192, most)), frame, left,
                       right, sinks, lengths, layout)
        else:
            Nq = rng.choice([1, _log(rng, 2, 64), _log(rng, 65, min(8192, most))])
            Nk = Nq + _log(rng, 1, min(32768, most))
            c = _window("", dtype, B, H, Hkv, d, Nq, Nk, frame, left, right, sinks, lengths,
                        layout)
    del c["name"]
    return c


def _lengths(case):
    """Keys of each sequence: all of them, or from all down to about a third."""
    most = case["most"] if case["op"] == "paged" else case["Nk"]
    B = case["B"]
    if case.get("lengths") == "full":
        return [most] * B
    return [max(1, most - (2 * most * b) // (3 * B) - (b % 7)) for b in range(B)]


def _starts(case):
    """Position of each sequence's first query: 0 where the queries are the whole
    sequence, else such that the last query is the newest token."""
    if case["op"] == "paged":
        return [n - 1 for n in _lengths(case)]
    return [0 if case["Nq"] == case["Nk"] else n - case["Nq"] for n in _lengths(case)]


# ------------------------------------------------------------------ inputs
def _normal(shape, g, dtype):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return x.to(_DTYPES[dtype])


def _tokens(case, H, N, g):
    """Unit normal tokens, with a code of period 64 along the positions that queries and
    keys share: nearby and repeated content raises the logits, as in video tokens."""
    d = case["d"]
    x = torch.randn((case["B"], H, N, d), generator=g, device="cuda", dtype=torch.float32)
    n = torch.arange(N, device="cuda", dtype=torch.float32)[:, None]
    i = torch.arange(d, device="cuda", dtype=torch.float32)[None, :]
    x += 0.5 * torch.sin(n * (2 * math.pi / 64) * (1 + i % 4) + i)
    return x.to(_DTYPES[case["dtype"]])


def _laid_out(x, layout):
    return x if layout == "bhnd" else x.transpose(1, 2).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op, B, H, Hkv, d = case["op"], case["B"], case["H"], case["Hkv"], case["d"]
    if op == "rotary":
        N, layout = case["N"], case["layout"]
        s["q"] = _laid_out(_normal((B, H, N, d), g, case["dtype"]), layout)
        s["k"] = _laid_out(_normal((B, Hkv, N, d), g, case["dtype"]), layout)
        # angular frequencies of each axis: base ** (-2i / width), positions interpolated
        # by `factor`
        dims = [int(a) for a in case["axes"].split(",")]
        s["dims"] = tuple(dims)
        freqs = [10000.0 ** (-2.0 * i / a) / case["factor"] for a in dims for i in range(a // 2)]
        s["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
        if len(dims) == 3:   # the clip's (frame, row, column); its first frame is `first`
            s["grid"] = _grid(case)
        return s
    lens = _lengths(case)
    if op == "paged":
        page = case["page"]
        pages = [-(-n // page) for n in lens]
        width = max(pages)
        total = sum(pages) + 3
        s["q"] = _normal((B, H, d), g, case["dtype"])
        s["k_pages"] = _normal((total, Hkv, page, d), g, case["dtype"])
        s["v_pages"] = _normal((total, Hkv, page, d), g, case["dtype"])
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
            if case["left"] >= 0:   # pages that the window has passed were given back
                first = max(0, (lens[b] - 1 - case["left"]) // page)
                kept = -(-case["sinks"] // page)
                if kept < first:
                    table[b, kept:first] = -1
        s["table"] = table
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        return s
    layout = case["layout"]
    Nq, Nk = case["Nq"], case["Nk"]
    q, k = _tokens(case, H, Nq, g), _tokens(case, Hkv, Nk, g)
    v = _normal((B, Hkv, Nk, d), g, case["dtype"])
    if op == "window":   # a cache's rows behind each sequence were never written
        for b, n in enumerate(lens):
            k[b, :, n:] = float("nan")
            v[b, :, n:] = float("nan")
    else:
        s["dout"] = _laid_out(_normal((B, H, Nq, d), g, case["dtype"]), layout)
    s["q"], s["k"], s["v"] = (_laid_out(x, layout) for x in (q, k, v))
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor(_starts(case), dtype=torch.int32, device="cuda")
    return s


def _grid(case):
    """(frames, rows, columns) of N tokens: the 720p latent's 45 x 80, or the largest
    rows x columns of the other grids that divides N."""
    for h, w in ((45, 80), (30, 52), (8, 8), (4, 5), (1, 3)):
        if case["N"] % (h * w) == 0:
            return (case["N"] // (h * w), h, w)
    return (case["N"], 1, 1)


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _OWN[case["op"]](s, case)
    return _PLAIN[case["op"]](s, case)


def _own_window(s, c):
    return _framework().window_attention(
        s["q"], s["k"], s["v"], window=(c["left"], c["right"]), sinks=c["sinks"],
        frame=c["frame"], lengths=s["lengths"], starts=s["starts"], layout=c["layout"])


def _own_train(s, c):
    ops = _framework()
    mask = dict(window=(c["left"], c["right"]), sinks=c["sinks"], frame=c["frame"],
                lengths=s["lengths"], starts=s["starts"], layout=c["layout"])
    out, lse = ops.window_attention(s["q"], s["k"], s["v"], return_lse=True, **mask)
    dq, dk, dv = ops.window_attention_backward(s["q"], s["k"], s["v"], out, lse, s["dout"],
                                               **mask)
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _own_paged(s, c):
    return _framework().paged_attention(
        s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"],
        window=(c["left"], c["right"]), sinks=c["sinks"], frame=c["frame"])


def _own_rotary(s, c):
    ops = _framework()
    call = ops.rotary_backward if c["backward"] else ops.rotary
    return call(s["q"], s["k"], s["freqs"], dims=s["dims"], style=c["style"],
                grid=s.get("grid"), start=c["first"], layout=c["layout"])


_OWN = {"window": _own_window, "train": _own_train, "paged": _own_paged, "rotary": _own_rotary}


# ------------------------------------------------------------------ plain forms
def _mask(lengths, starts, Nq, Nk, c):
    """[B, Nq, Nk]: which keys a query sees."""
    dev = lengths.device
    p = starts[:, None] + torch.arange(Nq, device=dev)[None, :]
    j = torch.arange(Nk, device=dev)[None, None, :]
    n = lengths[:, None, None]
    fq = (p // c["frame"])[:, :, None]
    fk = j // c["frame"]
    see = (j < n) & ((p >= 0) & (p < lengths[:, None]))[:, :, None]
    if c["right"] >= 0:
        see = see & (fk <= fq + c["right"])
    if c["left"] >= 0:
        see = see & ((fk >= fq - c["left"]) | (fk < c["sinks"]))
    return see


def _attend(q, k, v, see, scale):
    """q [B, Hkv, G, Nq, d], k and v [B, Hkv, Nk, d] in 32 bits -> out like q, the
    probabilities and the rows' log-sum-exp."""
    B, Hkv, G, Nq, d = q.shape
    s = torch.matmul(q.reshape(B, Hkv, G * Nq, d), k.transpose(-1, -2)).mul_(scale)
    s = s.view(B, Hkv, G, Nq, -1).masked_fill_(~see[:, None, None], float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    out = torch.matmul(p.view(B, Hkv, G * Nq, -1), v).view(B, Hkv, G, Nq, d)
    return out, p, lse


def _heads(x, layout):
    return (x if layout == "bhnd" else x.transpose(1, 2)).float()


def _plain_window(s, c, whole=False):
    q, k, v = (_heads(s[n], c["layout"]) for n in ("q", "k", "v"))
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    there = torch.arange(Nk, device=k.device)[None, None, :, None] < s["lengths"][:, None, None, None]
    v = torch.where(there, v, torch.zeros_like(v))
    see = _mask(s["lengths"], s["starts"], Nq, Nk, c)
    scale = 1 / math.sqrt(d)
    q = q.reshape(B, Hkv, H // Hkv, Nq, d)
    out, p, lse = _attend(q, k, v, see, scale)
    o = out.view(B, H, Nq, d)
    result = _laid_out(o, c["layout"]).to(s["q"].dtype)
    return (result, (q, k, v, out, p, lse, scale)) if whole else result


def _plain_train(s, c):
    result, (q, k, v, out, p, lse, scale) = _plain_window(s, c, whole=True)
    B, Hkv, G, Nq, d = q.shape
    do = _heads(s["dout"], c["layout"]).reshape(B, Hkv, G, Nq, d)
    rows = (B, Hkv, G * Nq)
    dv = torch.matmul(p.view(*rows, -1).transpose(-1, -2), do.reshape(*rows, d))
    ds = torch.matmul(do.reshape(*rows, d), v.transpose(-1, -2)).view(p.shape)
    ds -= (do * out).sum(dim=-1, keepdim=True)
    ds *= p
    ds = ds.view(*rows, -1)
    dq = torch.matmul(ds, k).mul_(scale).view(B, Hkv * G, Nq, d)
    dk = torch.matmul(ds.transpose(-1, -2), q.reshape(*rows, d)).mul_(scale)
    dq, dk, dv = (_laid_out(x, c["layout"]).to(s["q"].dtype) for x in (dq, dk, dv))
    return {"out": result, "lse": lse.reshape(B, Hkv * G, Nq), "dq": dq, "dk": dk, "dv": dv}


def _plain_paged(s, c):
    B, H, d = s["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    table = s["table"].clamp(min=0).long()
    k, v = (s[n][table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
            for n in ("k_pages", "v_pages"))
    lengths = s["lengths"]
    see = _mask(lengths, lengths - 1, 1, k.shape[2], c)
    q = s["q"].float().view(B, Hkv, H // Hkv, 1, d)
    out, _, _ = _attend(q, k, v, see, 1 / math.sqrt(d))
    return out.view(B, H, d).to(s["q"].dtype)


def _plain_rotary(s, c):
    N, dims, style = c["N"], s["dims"], c["style"]
    dev = s["q"].device
    n = torch.arange(N, device=dev, dtype=torch.float64)
    if len(dims) == 3:
        f, h, w = s["grid"]
        at = (c["first"] + (n / (h * w)).floor(), (n / w).floor() % h, n % w)
    else:
        at = (c["first"] + n,)
    axis = torch.cat([torch.full((a // 2,), i, device=dev) for i, a in enumerate(dims)])
    angle = torch.stack(at, dim=1)[:, axis] * s["freqs"]          # [N, pairs], 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    if c["backward"]:
        sin = -sin
    if c["layout"] == "bnhd":
        cos, sin = cos[:, None, :], sin[:, None, :]
    return [_turned(s[name], cos, sin, 2 * s["freqs"].numel(), style) for name in ("q", "k")]


def _turned(x, cos, sin, width, style):
    y = x.float()
    part, rest = y[..., :width], y[..., width:]
    if style == "interleaved":
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = part[..., :width // 2], part[..., width // 2:]
        part = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((part, rest), dim=-1).to(x.dtype)


_PLAIN = {"window": _plain_window, "train": _plain_train, "paged": _plain_paged,
          "rotary": _plain_rotary}


# ------------------------------------------------------------------ least work
def _reach(c, p, n):
    """(sink keys, first window key, end) that a query at position p of n keys sees."""
    fq = p // c["frame"]
    hi = n if c["right"] < 0 else min(n, (fq + c["right"] + 1) * c["frame"])
    lo = 0 if c["left"] < 0 else min(hi, max(0, fq - c["left"]) * c["frame"])
    return min(lo, c["sinks"] * c["frame"]), lo, hi


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    if case["op"] == "rotary":
        n = B * case["N"] * (H + Hkv)
        width = sum(int(a) for a in case["axes"].split(","))
        return {"bytes": 2 * n * d * size, "flops": 3 * n * width}
    Nq = 1 if case["op"] == "paged" else case["Nq"]
    pairs, keys = 0, 0
    for n, start in zip(_lengths(case), _starts(case)):
        first, last = max(0, start), min(n, start + Nq)
        if last <= first:
            continue
        # the rows of one frame see the same keys
        p, least, end, sink = first, None, 0, 0
        while p < last:
            stop = min(last, (p // case["frame"] + 1) * case["frame"])
            s, lo, hi = _reach(case, p, n)
            pairs += (stop - p) * (s + hi - lo)
            least = lo if least is None else min(least, lo)
            end, sink, p = max(end, hi), max(sink, s), stop
        keys += end - least + min(sink, least)
    q, kv = B * H * Nq * d * size, 2 * Hkv * keys * d * size
    if case["op"] == "train":
        # q, k, v, dout read and out, lse, dq, dk, dv written; two products forward, five
        # backward
        return {"bytes": 4 * q + 2 * kv + 4 * B * H * Nq, "flops": 14 * d * H * pairs}
    return {"bytes": 2 * q + kv, "flops": 4 * d * H * pairs}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s, case)
    if case["op"] == "paged":
        return _exact_paged(s, case)
    return _exact_window(s, case)


def _row_keys(c, lo_p, hi_p, n, dev):
    """Rows at positions lo_p .. hi_p - 1 of a sequence of n keys: their keys as a 0/1
    matrix."""
    see = torch.zeros((hi_p - lo_p, n), dtype=torch.bool, device=dev)
    rows = torch.arange(lo_p, hi_p, device=dev)
    cols = torch.arange(n, device=dev)
    fr = torch.div(rows, c["frame"], rounding_mode="floor")
    fc = torch.div(cols, c["frame"], rounding_mode="floor")
    dist = fr[:, None] - fc[None, :]
    see |= True
    if c["right"] >= 0:
        see &= dist >= -c["right"]
    if c["left"] >= 0:
        see &= (dist <= c["left"]) | (fc < c["sinks"])[None, :]
    return see


def _exact_head(q, k, v, see, scale):
    a = (q @ k.t()) * scale
    a[~see] = -math.inf
    lse = torch.logsumexp(a, dim=1)
    p = torch.exp(a - lse[:, None])
    p[lse == -math.inf] = 0
    return p, lse, p @ v


def _exact_window(s, c):
    B, H, Hkv, d, Nq, Nk = (c[n] for n in ("B", "H", "Hkv", "d", "Nq", "Nk"))
    dev = s["q"].device
    scale = d ** -0.5
    back = c["op"] == "train"

    def head(x, b, h):
        return (x[b, h] if c["layout"] == "bhnd" else x[b, :, h]).double()

    out = torch.zeros((B, H, Nq, d), dtype=torch.float64, device=dev)
    lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device=dev)
    dq = torch.zeros_like(out) if back else None
    dk = torch.zeros((B, Hkv, Nk, d), dtype=torch.float64, device=dev) if back else None
    dv = torch.zeros_like(dk) if back else None
    for b, (n, start) in enumerate(zip(_lengths(c), _starts(c))):
        lo_p, hi_p = max(0, start), min(n, start + Nq)
        if hi_p <= lo_p:
            continue
        rows = slice(lo_p - start, hi_p - start)
        see = _row_keys(c, lo_p, hi_p, n, dev)
        for h in range(H):
            g = h // (H // Hkv)
            q, k, v = head(s["q"], b, h)[rows], head(s["k"], b, g)[:n], head(s["v"], b, g)[:n]
            p, l, o = _exact_head(q, k, v, see, scale)
            out[b, h, rows], lse[b, h, rows] = o, l
            if back:
                do = head(s["dout"], b, h)[rows]
                dv[b, g, :n] += p.t() @ do
                dp = do @ v.t()
                da = p * (dp - (p * dp).sum(dim=1, keepdim=True))
                dq[b, h, rows] = scale * (da @ k)
                dk[b, g, :n] += scale * (da.t() @ q)
    out = _laid_out(out, c["layout"])
    if not back:
        return out
    dq, dk, dv = (_laid_out(x, c["layout"]) for x in (dq, dk, dv))
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _exact_paged(s, c):
    B, H, Hkv, d, page = c["B"], c["H"], c["Hkv"], c["d"], c["page"]
    dev = s["q"].device
    out = torch.zeros((B, H, d), dtype=torch.float64, device=dev)
    for b, n in enumerate(_lengths(c)):
        sink, lo, hi = _reach(c, n - 1, n)
        j = torch.cat((torch.arange(sink, device=dev), torch.arange(lo, hi, device=dev)))
        at = s["table"][b][j // page].long()
        for g in range(Hkv):
            k, v = (s[x][at, g, j % page].double() for x in ("k_pages", "v_pages"))
            heads = slice(g * (H // Hkv), (g + 1) * (H // Hkv))
            a = (s["q"][b, heads].double() @ k.t()) / math.sqrt(d)
            out[b, heads] = torch.softmax(a, dim=1) @ v
    return out


def _exact_rotary(s, c):
    N, dims = c["N"], s["dims"]
    dev = s["q"].device
    n = torch.arange(N, device=dev)
    if len(dims) == 3:
        _, h, w = s["grid"]
        at = [n // (h * w) + c["first"], n // w % h, n % w]
    else:
        at = [n + c["first"]]
    turn, first = [], 0
    for pos, a in zip(at, dims):
        turn.append(torch.outer(pos.double(), s["freqs"][first:first + a // 2]))
        first += a // 2
    turn = torch.cat(turn, dim=1)
    unit = torch.polar(torch.ones_like(turn), -turn if c["backward"] else turn)
    if c["layout"] == "bnhd":
        unit = unit[:, None, :]
    result = []
    for name in ("q", "k"):
        y = s[name].double()
        part = y[..., :2 * first]
        if c["style"] == "interleaved":
            z = torch.view_as_complex(part.unflatten(-1, (first, 2)).contiguous()) * unit
            part = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(part[..., :first], part[..., first:]) * unit
            part = torch.cat((z.real, z.imag), dim=-1)
        result.append(torch.cat((part, y[..., 2 * first:]), dim=-1))
    return result
