"""Plain binary64 attention with rules on the scores, for the tests, and the bounds that go with it.

Beside the bounds of attn_util (u = 2^-8 for the roundings to bf16, 2^-10 for what binary32 adds to
each weight), a rule adds to each weight:

* a cap: the tanh is off by at most 7e-6 (its fit with the roundings of binary32, or fewer units of
  2^-23), so a score moves by at most 8e-6 cap, and a weight, whose row's sum moves too, by twice
  that: 16e-6 cap.
* a distance bias: slope * distance rounds to 2^-24 of itself in the product, in up to eight sums from
  one column to the next, in the sum with the score, and once scaled by log2(e): 11 * 2^-24 * 1.45 *
  slope * distance, twice for the row's sum.  Keys
  whose weight counts at all (above 2^-24 of the largest) are those whose bias stays within 20 plus
  the scores' spread of the row's best; the bound takes the whole of it.

ds = p (1 - tanh^2) (dP - D): the factor's error, 2e-5 absolute where it is at least 0.36 and a few
2^-23 of its own terms beyond, stays below 2^-13 of it where it counts and is inside binary32's 2^-10
of the others.
"""
from __future__ import annotations

import math

import torch

from attn_util import B32, U, heads


def visible(n, m, causal, prefix, device):
    """Row i of n, at position m - n + i, sees key j of m: those up to its own, and the prefix."""
    i = torch.arange(n, device=device)[:, None] + (m - n)
    j = torch.arange(m, device=device)[None, :]
    seen = (j <= i) if causal else torch.ones((n, m), dtype=torch.bool, device=device)
    if prefix is not None and causal:
        seen = seen | (j < prefix)
    return seen & (i >= 0)


def scores(q, k, scale, cap, slopes, pos):
    """(scores, 1 - tanh^2) of heads-first binary64 q [H, n, d] and k [H, m, d]; pos: positions of
    the rows."""
    s = scale * (q @ k.transpose(1, 2))
    factor = torch.ones_like(s)
    if cap:
        t = torch.tanh(s / cap)
        s, factor = cap * t, 1.0 - t * t
    if slopes is not None:
        far = (pos[:, None] - torch.arange(k.shape[1], device=k.device)[None, :]).abs().double()
        s = s - slopes.double()[:, None, None] * far
    return s, factor


def sample_reference(q, k, v, scale, cap=0.0, slopes=None, prefix=None, causal=True, dout=None):
    """One sample: q [n, Hq, d], k, v [m, Hkv, d].  A dict of results (o, lse, and with dout dq, dk,
    dv), each as (value, bound), all [rows, heads, d]."""
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    g = hq // hkv
    Q, K, V = heads(q), heads(k, g), heads(v, g)
    pos = torch.arange(n, device=q.device) + (m - n)
    seen = visible(n, m, causal, prefix, q.device)
    s, factor = scores(Q, K, scale, cap, slopes, pos)
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(dim=2, keepdim=True) if m else s.new_full((hq, n, 1), -math.inf)
    top = torch.where(top.isfinite(), top, torch.zeros_like(top))
    e = torch.where(seen, torch.exp(s - top), torch.zeros_like(s))
    l = e.sum(dim=2, keepdim=True)
    p = e / torch.where(l > 0, l, torch.ones_like(l))
    steep = 0.0 if slopes is None else float(slopes.abs().max()) * m
    rule = 16e-6 * cap + 2 * 11 * 1.45 * 2.0 ** -24 * steep
    o = p @ V
    tol_o = U * o.abs() + (U + B32 + rule) * (p @ V.abs()) + 1e-30
    out = {"o": (o.transpose(0, 1), tol_o.transpose(0, 1)), "lse": (torch.log(l) + top)[:, :, 0], "rule": rule}
    if dout is None:
        return out
    G = heads(dout)
    dP = G @ V.transpose(1, 2)
    D = (G * o).sum(dim=2, keepdim=True)
    dD = (G.abs() * tol_o).sum(dim=2, keepdim=True)
    ds = p * factor * (dP - D)
    tol_ds = U * ds.abs() + p * factor * dD + (B32 + rule) * p * factor * (dP.abs() + D.abs())
    fold = lambda x: x.view(hkv, g, *x.shape[1:]).sum(dim=1)                          # noqa: E731
    dq, dk, dv = scale * (ds @ K), fold(scale * (ds.transpose(1, 2) @ Q)), fold(p.transpose(1, 2) @ G)
    for name, x, t in (("dq", dq, scale * (tol_ds @ K.abs())), ("dk", dk, fold(scale * (tol_ds.transpose(1, 2) @ Q.abs()))),
                       ("dv", dv, fold((U + B32 + rule) * (p.transpose(1, 2) @ G.abs())))):
        out[name] = (x.transpose(0, 1), (t + U * x.abs() + 1e-30).transpose(0, 1))
    return out
