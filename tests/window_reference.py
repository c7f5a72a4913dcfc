"""Plain 64-bit window attention and its gradients, with bounds on what the kernels'
roundings may add, element by element.

The bounds, with u = half a step of the type (torch.finfo.eps / 2: 2^-8 for bfloat16,
2^-24 for float32) and e an upper bound on the relative error of one probability in
32-bit arithmetic:
  logits   each is a sum of d products in float32, scaled and reduced by the row's
           maximum: at most (d + 4) 2^-24 scale |q|.|k| off, which is the relative error
           of its exponential, on top of 2^-21 for exp2 and the rounding of its argument
           (|argument| < 2^3 where the exponential matters)
  out      P rounded to the type: u P each, summed |v|; the sum of n terms in float32;
           the result rounded: u |out|
  delta    sum of dout * out with out as the forward gave it
  dS       P (dP - delta), rounded to the type: u |dS|
and the gradients are sums of those against |k|, |q|, |dout|, rounded to the type.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def visible(B, Nq, Nk, window, sinks, frame, lengths, starts, device):
    left, right = window
    n = torch.full((B,), Nk, device=device) if lengths is None else \
        lengths.long().clamp(0, Nk)
    s = n - Nq if starts is None else (
        torch.full((B,), starts, device=device) if isinstance(starts, int) else starts.long())
    pos = s[:, None] + torch.arange(Nq, device=device)
    j = torch.arange(Nk, device=device)
    see = ((pos >= 0) & (pos < n[:, None]))[:, :, None] & (j < n[:, None])[:, None, :]
    fq, fk = (pos // frame)[:, :, None], (j // frame)[None, None, :]
    if right >= 0:
        see = see & (fk <= fq + right)
    if left >= 0:
        see = see & ((fk >= fq - left) | (fk < sinks))
    return see


def attention(q, k, v, dout=None, *, window=(-1, 0), sinks=0, frame=1, lengths=None, starts=None,
              scale=None, layout="bhnd"):
    """dict of 64-bit out, lse (dq, dk, dv) and of the bounds on their errors."""
    u = U[q.dtype]
    sw = (lambda x: x) if layout == "bhnd" else (lambda x: x.transpose(1, 2))
    qd, kd, vd = (sw(x).double() for x in (q, k, v))
    B, H, Nq, d = qd.shape
    Hkv, Nk = kd.shape[1], kd.shape[2]
    G = H // Hkv
    see = visible(B, Nq, Nk, window, sinks, frame, lengths, starts, q.device)
    keep = see.any(dim=1)[:, None, :, None]           # keys that no query sees may be NaN
    kd, vd = torch.where(keep, kd, 0.0), torch.where(keep, vd, 0.0)
    real = see.any(dim=2)[:, None, :, None]           # and rows that see no key
    qd = torch.where(real, qd, 0.0)
    kg, vg = (x.repeat_interleave(G, dim=1) for x in (kd, vd))
    scale = 1 / math.sqrt(d) if scale is None else scale
    see = see[:, None]
    a = torch.where(see, qd @ kg.transpose(-1, -2) * scale, -math.inf)
    lse = torch.logsumexp(a, dim=-1)
    p = torch.where(see, (a - torch.where(lse == -math.inf, 0.0, lse)[..., None]).exp(), 0.0)
    out = p @ vg
    mag = torch.where(see, qd.abs() @ kg.abs().transpose(-1, -2) * scale, 0.0).amax()
    e = float((d + 4) * 2.0 ** -24 * mag + 2.0 ** -21)
    up = u if q.dtype == torch.bfloat16 else 2.0 ** -24
    n_sum = 2.0 ** -24 * 64                            # blocked sums
    absv = p @ vg.abs()
    out_err = (up + 2 * e + n_sum) * absv * 1.01 + u * out.abs()
    r = {"out": sw(out), "lse": lse, "out_bound": sw(out_err),
         "lse_bound": 2 * e + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)}
    if dout is None:
        return r
    do = torch.where(real, sw(dout).double(), 0.0)
    dp = do @ vg.transpose(-1, -2)
    delta = (do * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    fold = lambda x: x.view(B, Hkv, G, *x.shape[2:]).sum(2)   # noqa: E731
    dq = ds @ kg * scale
    dk = fold(ds.transpose(-1, -2) @ qd) * scale
    dv = fold(p.transpose(-1, -2) @ do)
    delta_err = (do.abs() * out_err).sum(-1, keepdim=True)
    dp_err = (d + 4) * 2.0 ** -24 * (do.abs() @ vg.abs().transpose(-1, -2))
    ds_err = (up + 2 * e) * ds.abs() + p * (delta_err + dp_err) * 1.01
    pr = (up + 2 * e + n_sum) * 1.01
    r["dq"], r["dk"], r["dv"] = sw(dq), sw(dk), sw(dv)
    r["dq_bound"] = sw((ds_err + n_sum * ds.abs()) @ kg.abs() * scale * 1.01 + u * dq.abs())
    r["dk_bound"] = sw(fold((ds_err + n_sum * ds.abs()).transpose(-1, -2) @ qd.abs()) * scale *
                       1.01 + u * dk.abs())
    r["dv_bound"] = sw(fold(pr * p.transpose(-1, -2) @ do.abs()) + u * dv.abs())
    return r


def assert_within(got, want, bound, name):
    got = got.double()
    assert got.shape == want.shape, name
    same_inf = torch.isinf(want) & (got == want)
    err = torch.where(same_inf, 0.0, (got - want).abs())
    slack = bound + 1e-30
    bad = ~(err <= slack)
    if bad.any():
        i = int(torch.nan_to_num(err / slack, nan=1e30).flatten().argmax())
        raise AssertionError("%s: %d of %d outside the bound; worst at %d: got %g want %g bound %g"
                             % (name, int(bad.sum()), bad.numel(), i, got.flatten()[i],
                                want.flatten()[i], slack.flatten()[i]))
