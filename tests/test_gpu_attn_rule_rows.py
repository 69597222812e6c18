"""What of other rows and keys a row's bits depend on under a rule (needs a GB300): not on keys that its warp
does not see; on the scores of its warp's rows as far as the forms of the tanh differ."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import assert_within, normal  # noqa: E402
from rule_bounds import tight  # noqa: E402
from test_gpu_attn_rules import dev, ints, pr, series  # noqa: E402, F401


RULES = {"cap": dict(score_cap=5.0), "cap-100": dict(score_cap=100.0), "cap-500": dict(score_cap=500.0), "slopes": {},
         "cap-slopes": dict(score_cap=9.0)}


def arguments(name, dev, hq):
    rule = dict(RULES[name])
    if "slopes" in name:
        rule["distance_slopes"] = series(hq, dev)
    return rule


@pytest.mark.parametrize("name", list(RULES))
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 1, 128)])
def test_keys_that_a_warp_does_not_see_change_no_bit(dev, name, hq, hkv, d):
    """Keys and values past the 32 rows of a warp, (token, head) pairs: out, lse and dq of the rows before."""
    m, n = pr(), 400
    q, k, v, dout = (normal((n, h, d), 70 + i, dev) for i, h in enumerate((hq, hkv, hkv, hq)))
    q *= 6
    cu, rule = ints([0, n], dev), arguments(name, dev, hq)
    tokens = 32 * hkv // hq

    def run(kk, vv):
        o, lse = m.attn_varlen_fwd(q, kk, vv, cu, return_lse=True, **rule)
        return o, lse, m.attn_varlen_bwd(dout, q, kk, vv, o, lse, cu, **rule)[0]

    o, lse, dq = run(k, v)
    for first in (tokens, 5 * tokens, 384):
        kk, vv = k.clone(), v.clone()
        kk[first:] = normal((n - first, hkv, d), 75, dev) * 300
        vv[first:] = -vv[first:] * 7
        o2, lse2, dq2 = run(kk, vv)
        assert torch.equal(o[:first], o2[:first]) and torch.equal(lse[:, :first], lse2[:, :first])
        whole = first // 32 * 32                     # (the backward's warps have 32 tokens of a head)
        assert torch.equal(dq[:whole], dq2[:whole])
        assert not torch.equal(o[first:], o2[first:])


@pytest.mark.parametrize("cap", [5.0, 50.0, 100.0])
def test_a_later_query_moves_an_earlier_row_by_the_forms_error_alone(dev, cap):
    """The form of the tanh is chosen by the scores of a warp's rows: the last one's query takes the others
    from the short form to another.  Both are within the bounds, so that they differ by twice those at most."""
    m, n = pr(), 96
    q, k, v = normal((n, 1, 64), 80, dev), normal((n, 1, 64), 81, dev), normal((n, 1, 64), 82, dev)
    cu = ints([0, n], dev)
    q *= 0.02 * cap
    o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True, score_cap=cap)
    other = q.clone()
    other[63] = k[3] * cap
    o2, lse2 = m.attn_varlen_fwd(other, k, v, cu, return_lse=True, score_cap=cap)
    assert torch.equal(o[:32], o2[:32]) and torch.equal(o[64:], o2[64:])
    ref = tight(q, k, v, 0.125, cap)
    rows = list(range(32, 63))
    for a, b, (value, tol) in ((o[rows], o2[rows], [x[rows] for x in ref["o"]]),
                               (lse[:, rows], lse2[:, rows], [x[:, rows] for x in ref["lse"]])):
        assert_within(a, value, tol, "before")
        assert_within(b, value, tol, "after")
        assert bool(((a.double() - b.double()).abs() <= 2 * tol).all())
