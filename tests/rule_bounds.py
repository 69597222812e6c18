"""Bounds of attention under a rule, score by score and row by row, for the tests (binary64).

rule_util bounds every weight of a call by its steepest slope, its longest distance and 16e-6 of the cap,
which says little of large caps and of slopes.  Here each score s_ij = u_ij (capped, biased) has its own
error, and a weight p_ij, relative to itself, is off by

    e_ij + sum_j p_ij e_ij        (its own score's error, and through the row's sum)

* the product: d multiplications added in binary32, each addition off by at most a unit in the last
  place: d 2^-23 of A_ij = scale sum |q||k|; a cap passes on at most as much.
* scale, cap and log2(e) as binary32 numbers and products with them: 2^-21 of the score.
* a cap up to 128: 8e-6 of it (its tanh is off by 7e-6).  A cap past 128: 1e-6 of the score where that is
  below the cap, else 2^-21 of the cap.
* a bias: the slope times log2(e), its product with the distance, up to eight sums from one column to the
  next and the one with the score round to 2^-24 each.  The sums start at a column up to 15 before the key's,
  so that none of them is of more than slope (|i - j| + 15) + |m| with m the row's maximum, which is folded
  in, and an error made there stays in the sums after it: 11 2^-24 (slope_h (|i - j| + 15) + |m_i|).
* the exponent's last sum and the exponential: 2^-22 (|s_ij| + |m_i|) + 2^-21.

lse is off by sum_j p_ij e_ij, by the sum in binary32, 2^-24 a key, and by its own roundings, 2^-22 (|lse| + |m|).
o adds one rounding of the result and of each weight to bf16, u = 2^-8, and the accumulation in binary32,
2^-24 a key of sum p |v|.  Where the result is divided by the sum of the weights as rounded (caps up to 55),
sum p delta (v - o) takes the place of sum p delta v: u |o| more.
"""
from __future__ import annotations

import math

import torch

from attn_util import U, heads
from rule_util import scores, visible


def tight(q, k, v, scale, cap=0.0, slopes=None, prefix=None, causal=True):
    """One sample: {"o": (value, bound) [rows, heads, d], "lse": (value, bound) [heads, rows], "p": weights}."""
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    g = hq // hkv
    Q, K, V = heads(q), heads(k, g), heads(v, g)
    pos = torch.arange(n, device=q.device) + (m - n)
    seen = visible(n, m, causal, prefix, q.device)
    s, _ = scores(Q, K, scale, cap, slopes, pos)
    u = scale * (Q @ K.transpose(1, 2))
    e = d * 2.0 ** -23 * scale * (Q.abs() @ K.abs().transpose(1, 2)) + 2.0 ** -21 * u.abs()
    if cap:
        capped = cap * torch.tanh(u / cap)
        e = torch.minimum(e, torch.full_like(e, 2 * cap))
        e = e + (8e-6 * cap if cap <= 128 else torch.where(u.abs() <= cap, 1e-6 * capped.abs(), torch.full_like(u, 2.0 ** -21 * cap)))
    top = torch.where(seen, s, torch.full_like(s, -math.inf)).amax(dim=2, keepdim=True)
    if slopes is not None:
        far = (pos[:, None] - torch.arange(m, device=k.device)[None, :]).abs().double()
        e = e + 11 * 2.0 ** -24 * (slopes.double().abs()[:, None, None] * (far + 15) + top.abs())
    e = e + 2.0 ** -22 * (s.abs() + top.abs()) + 2.0 ** -21
    w = torch.where(seen, torch.exp(s - top), torch.zeros_like(s))
    l = w.sum(dim=2, keepdim=True)
    p = w / l
    off = (p * e).sum(dim=2, keepdim=True)
    keys = seen.sum(dim=1)[None, :, None].double()
    o = p @ V
    divided = 1 if cap and cap <= 55.0 and slopes is None else 0
    tol = (1 + divided) * U * o.abs() + (p * (U + e + off + keys * 2.0 ** -24)) @ V.abs() + 1e-30
    lse = (torch.log(l) + top)[:, :, 0]
    tol_lse = (off + keys * 2.0 ** -24 + 2.0 ** -22 * top.abs())[:, :, 0] + 2.0 ** -22 * (lse.abs() + 1)
    return {"o": (o.transpose(0, 1), tol.transpose(0, 1)), "lse": (lse, tol_lse), "p": p}
