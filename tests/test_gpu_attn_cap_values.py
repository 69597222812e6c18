"""Capped scores and values far from 1 (needs a GB300): whatever the scores' place between -cap and cap,
finite values give the definition's result, within the bounds of any other values."""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import assert_within, normal  # noqa: E402
from rule_util import sample_reference  # noqa: E402
from test_gpu_attention import make_paged  # noqa: E402
from test_gpu_attn_rules import dev, ints, pr  # noqa: E402, F401

SIZES = [1e-22, 1e-12, 1e13, 1e20, 1e30]


def rows_at(kinds, n, hq, d, dev):
    """Queries whose scores against ``keys_at`` (scale 1/8) are about kinds[i % len] times 20 d."""
    sign = torch.tensor(kinds, device=dev).repeat(-(-n // len(kinds)))[:n]
    return (sign[:, None, None] * 40.0).expand(n, hq, d).to(torch.bfloat16).contiguous()


def keys_at(n, hkv, d, dev, seed=53):
    return (4.0 + normal((n, hkv, d), seed, dev).float() / 16).to(torch.bfloat16)


def close(o, lse, ref, what):
    assert_within(o, *ref["o"], what)
    if lse is not None:
        assert float((lse.double() - ref["lse"]).abs().max()) <= ref["rule"] + 2.0 ** -11 * (1 + float(ref["lse"].abs().max()))


# all rows near the cap, all near its negative, rows of all kinds side by side
KINDS = [(1.0,), (-1.0,), (1.0, -1.0, 0.001, -0.02)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("kinds", KINDS, ids=str)
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (4, 4, 128), (6, 2, 80)])
def test_packed(dev, hq, hkv, d, kinds, size):
    m = pr()
    lengths = [400, 1, 90, 900]
    T = sum(lengths)
    q, k, v = rows_at(kinds, T, hq, d, dev), keys_at(T, hkv, d, dev), (normal((T, hkv, d), 54, dev).float() * size).to(torch.bfloat16)
    cu = [0, 400, 401, 491, T]
    for cap in (30.0, 50.0, 55.0, 56.0):
        o, lse = m.attn_varlen_fwd(q, k, v, ints(cu, dev), scale=0.125, score_cap=cap, return_lse=True)
        for a, b in zip(cu, cu[1:]):
            ref = sample_reference(q[a:b], k[a:b], v[a:b], 0.125, cap)
            close(o[a:b], lse[:, a:b], ref, "cap %g, rows %d..%d" % (cap, a, b))
    assert not m.attn_fault()


@pytest.mark.parametrize("kinds", KINDS, ids=str)
def test_one_column_far_from_the_others(dev, kinds):
    """Values near 1 but for one column, tiny or huge; columns of zeros among them."""
    m, n = pr(), 300
    q, k, v = rows_at(kinds, n, 2, 128, dev), keys_at(n, 1, 128, dev), normal((n, 1, 128), 55, dev)
    v[:, :, 40:44] = 0
    for column in (0, 100):
        for size in (1e-24, 1e28):
            w = v.clone()
            w[:, :, column] = (w[:, :, column].float() * size).to(torch.bfloat16)
            o, lse = m.attn_varlen_fwd(q, k, w, ints([0, n], dev), scale=0.125, score_cap=55.0, return_lse=True)
            close(o, lse, sample_reference(q, k, w, 0.125, 55.0), "column %d, %g" % (column, size))


@pytest.mark.parametrize("size", [1e-22, 1.0, 1e30])
@pytest.mark.parametrize("new,kv,pages", [([300], [12000], 0), ([40, 200], [9000, 700], 0), ([130], [1000], 700)], ids=str)
def test_paged(dev, new, kv, pages, size):
    """Chunks, with the keys split and whole."""
    m = pr()
    cache, table, k_of, v_of = make_paged(dev, kv, 64, 1, 64, 7)
    for p, c in ((cache.k_pages, lambda x: 4.0 + x.float() / 16), (cache.v_pages, lambda x: x.float() * size)):
        p.copy_(torch.where(p.isfinite(), c(p), p.float()).to(torch.bfloat16))
    k_of, v_of = [(4.0 + x.float() / 16).to(torch.bfloat16) for x in k_of], [(x.float() * size).to(torch.bfloat16) for x in v_of]
    if pages:
        table = torch.cat([table, torch.full((len(kv), pages), 1 << 30, dtype=torch.int32, device=dev)], dim=1)
    T = sum(new)
    q = rows_at(KINDS[2], T, 2, 64, dev)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    o = m.attn_paged(q, cache, table, ints(kv, dev), ints(cu, dev), scale=0.125, score_cap=55.0)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        close(o[a:b], None, sample_reference(q[a:b], k_of[i], v_of[i], 0.125, 55.0), "rows %d..%d" % (a, b))
    assert not m.attn_fault()


@pytest.mark.parametrize("size", [1e-22, 1e30])
def test_other_rows_keep_their_bits(dev, size):
    """Rows of ordinary scores, with rows of scores at the caps in other warps of their tile and without."""
    m, n = pr(), 256
    q, k = normal((n, 1, 64), 56, dev), normal((n, 1, 64), 57, dev)
    v = (normal((n, 1, 64), 58, dev).float() * size).to(torch.bfloat16)
    cu = ints([0, n], dev)
    want = m.attn_varlen_fwd(q, k, v, cu, score_cap=50.0)
    for rows in (slice(32, 64), slice(200, 224)):
        far = q.clone()
        far[rows] = k[:1] * 400.0
        other = torch.ones(n, dtype=torch.bool, device=dev)
        other[rows.start // 32 * 32:-(-rows.stop // 32) * 32] = False
        got = m.attn_varlen_fwd(far, k, v, cu, score_cap=50.0)
        assert torch.equal(got[other], want[other])
        assert_within(got, *sample_reference(far, k, v, 0.125, 50.0)["o"], "o")


def test_infinite_values_come_out(dev):
    """A value of infinity is its rows' result (and NaN where it meets its negative), not another one's."""
    m, n = pr(), 200
    q, k, v = rows_at(KINDS[2], n, 1, 64, dev), keys_at(n, 1, 64, dev), normal((n, 1, 64), 59, dev)
    v[50, 0, 3], v[90, 0, 5] = math.inf, -math.inf
    o = m.attn_varlen_fwd(q, k, v, ints([0, 100, n], dev), scale=0.125, score_cap=50.0)
    assert bool((o[50:100, 0, 3] == math.inf).all()) and bool((o[90:100, 0, 5] == -math.inf).all())
    assert bool(o[100:].isfinite().all())
    keep = [c for c in range(64) if c not in (3, 5)]
    w = v.clone()
    w[50, 0, 3] = w[90, 0, 5] = 0
    ref = sample_reference(q[:100], k[:100], w[:100], 0.125, 50.0)
    assert_within(o[:100, :, keep], *(x[:, :, keep] for x in ref["o"]), "o")
