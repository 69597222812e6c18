"""Attention under a rule against bounds of its own for every score and row (needs a GB300): large caps
keep the precision of small scores, a bias is exact in every head and at every distance, lse is binary32's."""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import assert_within, normal, offsets  # noqa: E402
from rule_bounds import tight  # noqa: E402
from test_gpu_attention import make_paged, qkv_views  # noqa: E402
from test_gpu_attn_rules import dev, ints, pr, series  # noqa: E402, F401


def check_varlen(dev, lengths, hq, hkv, d, qscale, cap=0.0, slopes=None, prefix=None, causal=True, seed=1):
    m, cu = pr(), offsets(lengths)
    q, k, v = qkv_views(cu[-1], hq, hkv, d, seed, dev, "fused")
    q.mul_(qscale)
    scale = 1 / math.sqrt(d)
    o, lse = m.attn_varlen_fwd(q, k, v, ints(cu, dev), causal=causal, return_lse=True, score_cap=cap, distance_slopes=slopes,
                               prefix_lens=None if prefix is None else ints(prefix, dev))
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        ref = tight(q[a:b], k[a:b], v[a:b], scale, cap, slopes, None if prefix is None else prefix[i], causal)
        assert_within(o[a:b], *ref["o"], "o of rows %d..%d" % (a, b))
        assert_within(lse[:, a:b], *ref["lse"], "lse of rows %d..%d" % (a, b))


def check_paged(dev, new, kv, hq, hkv, d, qscale, cap=0.0, slopes=None, seed=2):
    m = pr()
    cache, table, k_of, v_of = make_paged(dev, kv, 64, hkv, d, seed)
    cu = offsets(new)
    q = normal((cu[-1], hq, d), seed + 5, dev) * qscale
    o = m.attn_paged(q, cache, table, ints(kv, dev), ints(cu, dev), score_cap=cap, distance_slopes=slopes)
    for i, (a, b) in enumerate(zip(cu, cu[1:])):
        assert_within(o[a:b], *tight(q[a:b], k_of[i], v_of[i], 1 / math.sqrt(d), cap, slopes)["o"], "rows %d..%d" % (a, b))


@pytest.mark.parametrize("cap", [0.25, 5.0, 50.0, 100.0, 128.0, 129.0, 200.0, 1000.0, 2e4])
@pytest.mark.parametrize("qscale", [0.1, 5.0, 40.0, 400.0])
def test_caps(dev, cap, qscale):
    check_varlen(dev, [260, 90], 4, 2, 64, qscale, cap, seed=50)
    check_varlen(dev, [300], 2, 1, 128, qscale, cap, causal=False, seed=51)


@pytest.mark.parametrize("cap", [50.0, 200.0, 1000.0, 2e4])
@pytest.mark.parametrize("qscale", [5.0, 40.0])
def test_caps_paged(dev, cap, qscale):
    check_paged(dev, [1, 1, 1], [900, 1, 90], 8, 2, 128, qscale, cap)
    check_paged(dev, [150, 40], [400, 90], 4, 2, 64, qscale, cap)


@pytest.mark.parametrize("first", [0.0, -0.01, 0.02, 0.5, 4.0, 40.0])
@pytest.mark.parametrize("causal", [True, False])
def test_slopes(dev, first, causal):
    check_varlen(dev, [700, 130], 4, 4, 64, 1.5, slopes=series(4, dev, first), causal=causal, seed=52)
    check_varlen(dev, [1500], 8, 2, 128, 1.5, slopes=series(8, dev, first), causal=causal, seed=53)
    check_varlen(dev, [700], 4, 2, 80, 6.0, 20.0, slopes=series(4, dev, first), causal=causal, seed=54)
    if causal:
        check_varlen(dev, [700, 130], 4, 4, 64, 1.5, slopes=series(4, dev, first), prefix=[300, 5], seed=55)


@pytest.mark.parametrize("first", [-0.01, 0.02, 0.5, 4.0])
def test_slopes_paged(dev, first):
    check_paged(dev, [1, 1, 1], [2900, 1, 90], 8, 2, 128, 1.5, slopes=series(8, dev, first))
    check_paged(dev, [1, 3], [9000, 300], 4, 1, 64, 6.0, 30.0, slopes=series(4, dev, first))
    check_paged(dev, [150, 40], [1400, 90], 4, 2, 64, 1.5, slopes=series(4, dev, first))
