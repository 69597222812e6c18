"""Gradients of sharp uncapped scores under a rule (needs a GB300): the accuracy that the header states."""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import normal, offsets  # noqa: E402
from rule_bounds import tight  # noqa: E402
from rule_util import sample_reference  # noqa: E402
from test_gpu_attn_rules import dev, ints, pr, series  # noqa: E402, F401


@pytest.mark.parametrize("lengths,hq,hkv,d", [([1500], 8, 2, 128), ([130, 300, 900], 4, 4, 64), ([700, 1, 450], 4, 1, 80)], ids=str)
@pytest.mark.parametrize("rule", ["slopes", "prefix"])
@pytest.mark.parametrize("qscale", [1.5, 6.0])
def test_gradients_of_sharp_uncapped_scores(dev, lengths, hq, hkv, d, rule, qscale):
    """Rounding to bf16 is off by 1.66e-3 of a value (mean square, 2^-8 / sqrt(3) of its binade, mantissas
    spread evenly over their logarithm).  Of dq and dk that is one rounding of the result and one of every
    ds; where D comes as dout . out, also p_ij times the error of that: d roundings of out, dout out each, and
    those of the weights p_ij that out is made of, p_ij dP_ij each, as out = sum p (1 + delta) v is off by sum p delta v
    and dout . v = dP.  So it is with dq under both rules, and with dk under a prefix alone, as the pass over the queries
    makes D whole for a biased dk.  All independent: their squares add up.  15 % for the statistics and
    binary32."""
    m, cu = pr(), offsets(lengths)
    q, k, v, dout = (normal((cu[-1], h, d), 90 + i, dev) for i, h in enumerate((hq, hkv, hkv, hq)))
    q *= qscale
    scale, step = 1 / math.sqrt(d), 1.66e-3
    slopes = series(hq, dev) if rule == "slopes" else None
    prefix = [n // 3 for n in lengths] if rule == "prefix" else None
    args = dict(distance_slopes=slopes, prefix_lens=None if prefix is None else ints(prefix, dev))
    o, lse = m.attn_varlen_fwd(q, k, v, ints(cu, dev), return_lse=True, **args)
    got = dict(zip(("dq", "dk"), m.attn_varlen_bwd(dout, q, k, v, o, lse, ints(cu, dev), **args)))
    want, wrong, expected = {"dq": 0.0, "dk": 0.0}, {"dq": 0.0, "dk": 0.0}, {"dq": 0.0, "dk": 0.0}
    g = hq // hkv
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        pre = None if prefix is None else prefix[i]
        ref = sample_reference(q[a:b], k[a:b], v[a:b], scale, 0.0, slopes, pre, True, dout[a:b])
        p = tight(q[a:b], k[a:b], v[a:b], scale, 0.0, slopes, pre)["p"]                      # [hq, n, n]
        Q, G = (x[a:b].double().transpose(0, 1) for x in (q, dout))
        K, V = (x[a:b].double().transpose(0, 1).repeat_interleave(g, 0) for x in (k, v))
        O = ref["o"][0].transpose(0, 1)
        dP = G @ V.transpose(1, 2)
        ds = p * (dP - (G * O).sum(2, keepdim=True))
        dD = ((step * G * O) ** 2).sum(2) + ((step * p * dP) ** 2).sum(2)                     # squared, of a row
        fold = lambda x: x.view(hkv, g, *x.shape[1:]).sum(1)                                 # noqa: E731
        var = {"dq": (step * ds) ** 2 @ K ** 2 + dD[..., None] * (p @ K) ** 2,
               "dk": fold(((step * ds) ** 2).transpose(1, 2) @ Q ** 2 +
                          ((p ** 2).transpose(1, 2) @ (dD[..., None] * Q ** 2) if rule == "prefix" else 0.0))}
        for name in want:
            x = ref[name][0]
            want[name] += float((x ** 2).sum())
            wrong[name] += float(((got[name][a:b].double() - x) ** 2).sum())
            expected[name] += float((scale ** 2 * var[name]).sum() + ((step * x) ** 2).sum())
    for name in want:
        err, limit = math.sqrt(wrong[name] / want[name]), 1.15 * math.sqrt(expected[name] / want[name])
        assert err <= limit, (name, err, limit)
        assert err <= (2.8e-3 if qscale == 1.5 else 5.0e-3)                                  # as include/attn.h has it
