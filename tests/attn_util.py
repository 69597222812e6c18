"""Plain binary64 attention for the tests, and the error bounds that go with it.

Bounds.  u = 2^-8 is the unit roundoff of bf16 (8 significant bits).  With p the weights
and everything else in binary64:

* o: one rounding of the result, u |o|, and one of each weight, u sum_j p |v|; what binary32
  adds (scores of up to 128 products: relative 2^-17 of sum |q||k| in the exponent, for the
  magnitudes used here at most 2^-11 of each weight) is bounded by 2^-10 sum_j p |v|.
* dv: the same with the sums over rows.
* dq, dk: one rounding of the result, one of each ds (u |ds|), the error of
  D = dout . o through the o it is given (each element within o's own bound), which enters
  every ds as p |error of D|, and binary32's part, 2^-10 p (|dP| + |D|).
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8
B32 = 2.0 ** -10


def heads(x, group=1):
    """[tokens, heads, d] -> float64 [heads * group, tokens, d]."""
    return x.double().transpose(0, 1).repeat_interleave(group, dim=0)


def sample_reference(q, k, v, scale, seen, dout=None):
    """One sample: q [n, Hq, d], k, v [m, Hkv, d], seen bool [n, m].  A dict of results
    (o, lse, and with dout dq, dk, dv), each as (value, bound), all [rows, heads, d]."""
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    g = hq // hkv
    Q, K, V = heads(q), heads(k, g), heads(v, g)
    s = scale * (Q @ K.transpose(1, 2))
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(dim=2, keepdim=True) if m else s.new_full((hq, n, 1), -math.inf)
    e = torch.where(seen, torch.exp(s - torch.where(top.isfinite(), top, torch.zeros_like(top))), torch.zeros_like(s))
    l = e.sum(dim=2, keepdim=True)
    p = e / torch.where(l > 0, l, torch.ones_like(l))
    o = p @ V
    tol_o = U * o.abs() + (U + B32) * (p @ V.abs()) + 1e-30
    lse = (torch.log(l) + top)[:, :, 0]
    out = {"o": (o.transpose(0, 1), tol_o.transpose(0, 1)), "lse": lse}
    if dout is None:
        return out
    G = heads(dout)
    dP = G @ V.transpose(1, 2)
    D = (G * o).sum(dim=2, keepdim=True)
    dD = (G.abs() * tol_o).sum(dim=2, keepdim=True)
    ds = p * (dP - D)
    tol_ds = U * ds.abs() + p * dD + B32 * p * (dP.abs() + D.abs())
    fold = lambda x: x.view(hkv, g, *x.shape[1:]).sum(dim=1)                          # noqa: E731
    dq, dk, dv = scale * (ds @ K), fold(scale * (ds.transpose(1, 2) @ Q)), fold(p.transpose(1, 2) @ G)
    for name, x, t in (("dq", dq, scale * (tol_ds @ K.abs())), ("dk", dk, fold(scale * (tol_ds.transpose(1, 2) @ Q.abs()))),
                       ("dv", dv, fold((U + B32) * (p.transpose(1, 2) @ G.abs())))):
        out[name] = (x.transpose(0, 1), (t + U * x.abs() + 1e-30).transpose(0, 1))
    return out


def causal_mask(n, m, causal, device):
    """Row i of n sees key j of m: j <= i + m - n, or all."""
    i = torch.arange(n, device=device)[:, None]
    j = torch.arange(m, device=device)[None, :]
    return (j <= i + (m - n)) if causal else torch.ones((n, m), dtype=torch.bool, device=device)


def assert_within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), "%s: %d of %d outside the bound, worst %.3g over %.3g" % (
        what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(nan=math.inf).max()), 1.0)


def normal(shape, seed, device, scale=1.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=device) * scale).to(torch.bfloat16)


def offsets(lengths, start=0):
    out = [start]
    for n in lengths:
        out.append(out[-1] + n)
    return out
