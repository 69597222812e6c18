"""The bounds of rule_bounds hold mistakes apart from rounding (no GPU): kernels' arithmetic restated in
numpy stays within them, the same with a mistake in it does not."""
from __future__ import annotations

import os
import re
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from rule_bounds import tight  # noqa: E402

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_varlen_rope_gb300", "csrc")


def constants(name, n):
    text = open(os.path.join(CSRC, "score_rule.cuh")).read()
    return [float(re.search(r"%s%d = ([-0-9.e]+)f" % (name, i), text).group(1)) for i in range(n)]


def odd(c, u):
    p = np.zeros_like(u)
    for x in c[::-1]:
        p = p * u * u + x
    return u * p


def large(u):
    """The form of caps past 128, in binary64."""
    return np.where(np.abs(u) <= 1, odd(constants("kTanh", 6), u), 1 - 2 / (1 + np.exp(2 * u)))


def short(u):
    """The forms of caps up to 128, as a mistake."""
    near = np.where(np.abs(u) <= 0.5, odd(constants("kSmall", 3), u), odd(constants("kNear", 4), u))
    return np.where(np.abs(u) <= 0.8, near, 1 - 2 / (1 + np.exp(2 * u)))


def restated(q, k, v, scale, cap, slopes, tanh=None, distance=lambda far: far, head=lambda h: h):
    """Attention of a causal sample with the weights rounded to bf16: (o [n, H, d], lse [H, n])."""
    n, hq, _ = q.shape
    g = hq // k.shape[1]
    outs, lses = [], []
    for h in range(hq):
        s = scale * (q[:, h].double() @ k[:, h // g].double().t()).numpy()
        if cap:
            s = cap * tanh(s / cap)
        if slopes is not None:
            i, j = np.ogrid[:n, :n]
            s = s - float(slopes[head(h)]) * distance(np.abs(i - j))
        s = torch.from_numpy(np.where(np.tril(np.ones((n, n), bool)), s, -np.inf))
        lse = torch.logsumexp(s, 1)
        p = torch.exp(s - s.amax(1, keepdim=True))
        l = p.sum(1, keepdim=True)
        outs.append(((p.float().bfloat16().double() @ v[:, h // g].double()) / l).float().bfloat16())
        lses.append(lse)
    return torch.stack(outs, 1), torch.stack(lses)


def outside(got, ref):
    """Worst multiple of the bound, of o and of lse."""
    o, lse = got
    return (float(((o.double() - ref["o"][0]).abs() / ref["o"][1]).max()),
            float(((lse - ref["lse"][0]).abs() / ref["lse"][1]).max()))


def tensors(n, hq, hkv, d, qscale, seed=1):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(n, h, d, generator=g) for h in (hq, hkv, hkv))
    return (q * qscale).bfloat16(), k.bfloat16(), v.bfloat16()


@pytest.mark.parametrize("cap", [200.0, 1000.0, 2e4])
@pytest.mark.parametrize("qscale", [5.0, 40.0])
def test_large_caps(cap, qscale):
    q, k, v = tensors(260, 2, 1, 64, qscale)
    ref = tight(q, k, v, 0.125, cap)
    assert max(outside(restated(q, k, v, 0.125, cap, None, large), ref)) <= 1.0
    if cap >= 1000:           # (6e-6 of a cap of 200 is 1.2e-3, what binary32's products may be off by here)
        assert outside(restated(q, k, v, 0.125, cap, None, short), ref)[1] > 2.0


@pytest.mark.parametrize("first", [0.5, 4.0, -0.02])
def test_slopes(first):
    q, k, v = tensors(300, 4, 2, 64, 1.5)
    slopes = torch.tensor([first * 2.0 ** (-7.5 * h / 4) for h in range(4)])
    ref = tight(q, k, v, 0.125, 0.0, slopes)
    assert max(outside(restated(q, k, v, 0.125, 0.0, slopes), ref)) <= 1.0
    for mistake in (dict(distance=lambda far: far + 1), dict(distance=lambda far: np.minimum(far, 127)),
                    dict(distance=lambda far: far * (1 + 2.0 ** -8)), dict(head=lambda h: h ^ 1)):
        assert max(outside(restated(q, k, v, 0.125, 0.0, slopes, **mistake), ref)) > 2.0, mistake
