"""Attention with capped scores, a bias by distance and prefixes against the binary64 definition
(needs a GB300): packed, with gradients, and over a paged cache."""
from __future__ import annotations

import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import B32, U, assert_within, normal, offsets  # noqa: E402
from rule_util import sample_reference  # noqa: E402
from test_gpu_attention import make_paged, qkv_views  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from packed_varlen_rope_gb300 import build

    build.build()
    return torch.device("cuda:0")


def pr():
    import packed_varlen_rope_gb300 as m

    return m


def ints(x, dev, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=dev)


def series(hq, dev, first=0.5):
    return torch.tensor([first * 2.0 ** (-7.5 * h / hq) for h in range(hq)], device=dev)


def check_varlen(dev, lengths, hq, hkv, d, cap=0.0, slopes=None, prefix=None, causal=True, layout="fused", used=None,
                 lead=0, tail=0, seed=1, scale=None, grads=True, qscale=1.5):
    m = pr()
    cu_list = offsets(lengths, lead)
    T = cu_list[-1] + tail
    q, k, v = qkv_views(T, hq, hkv, d, seed, dev, layout)
    q.mul_(qscale)
    dout = normal((T, hq, d), seed + 9, dev)
    used = list(lengths) if used is None else list(used)
    inside = torch.zeros(T, dtype=torch.bool, device=dev)
    for a, n in zip(cu_list, used):
        inside[a:a + n] = True
    for x in (q, k, v, dout):                                # other samples, padding: nothing may be read there
        x[~inside] = float("nan")
    cu = ints(cu_list, dev)
    rule = dict(causal=causal, scale=scale, seq_used=ints(used, dev) if used != list(lengths) else None, score_cap=cap,
                distance_slopes=slopes, prefix_lens=None if prefix is None else ints(prefix, dev))
    o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True, **rule)
    assert torch.equal(o, m.attn_varlen_fwd(q, k, v, cu, **rule))
    got = {"o": o}
    if grads:
        got.update(zip(("dq", "dk", "dv"), m.attn_varlen_bwd(dout, q, k, v, o, lse, cu, **rule)))
        again = m.attn_varlen_bwd(dout, q, k, v, o, lse, cu, **rule)
        assert all(torch.equal(got[n], x) for n, x in zip(("dq", "dk", "dv"), again))     # the same bits each run
    torch.cuda.synchronize()
    sc = 1 / math.sqrt(d) if scale is None else scale
    for i, (a, n) in enumerate(zip(cu_list, used)):
        if n == 0:
            continue
        ref = sample_reference(q[a:a + n], k[a:a + n], v[a:a + n], sc, cap, slopes, None if prefix is None else prefix[i],
                               causal, dout[a:a + n] if grads else None)
        for name, x in got.items():
            assert_within(x[a:a + n], *ref[name], "%s of rows %d..%d" % (name, a, a + n))
        err = (lse[:, a:a + n].double() - ref["lse"]).abs()
        assert float(err.max()) <= ref["rule"] + 2.0 ** -11 * (1 + float(ref["lse"].abs().max()))
    for name, x in got.items():
        assert not bool(x[~inside].any()), name + " of rows outside is not zero"
    assert bool((lse[:, ~inside] == -math.inf).all())
    assert not m.attn_fault()


RULES = {"cap": dict(cap=5.0), "slopes": dict(slopes=True), "prefix": dict(prefix=True), "cap-slopes": dict(cap=3.0, slopes=True),
         "all": dict(cap=20.0, slopes=True, prefix=True)}


def rule_for(name, lengths, hq, dev, seed=0):
    rng = random.Random("%s %s %d" % (name, lengths, seed))
    rule = dict(RULES[name])
    if rule.get("slopes"):
        rule["slopes"] = series(hq, dev)
    if rule.get("prefix"):
        rule["prefix"] = [rng.choice([0, 1, n // 2, n, n + 100, -5, rng.randint(0, max(n, 1)), 128, 129]) for n in lengths]
    return rule


LENGTHS = [[1], [2, 0, 1], [5, 17, 33, 9], [64, 64], [127, 1, 128, 129], [300, 0, 0, 255, 1], [513], [1000, 37]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("name", list(RULES))
def test_lengths(dev, name, lengths):
    check_varlen(dev, lengths, 4, 2, 64, lead=3, tail=5, **rule_for(name, lengths, 4, dev))
    check_varlen(dev, lengths, 8, 2, 128, seed=3, **rule_for(name, lengths, 8, dev, 1))


@pytest.mark.parametrize("name", ["cap", "slopes", "cap-slopes"])
@pytest.mark.parametrize("lengths", [[1], [127, 1, 128, 129], [700]], ids=str)
def test_both_directions(dev, name, lengths):
    check_varlen(dev, lengths, 6, 3, 80, causal=False, lead=1, tail=2, seed=5, **rule_for(name, lengths, 6, dev))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (14, 2), (16, 1), (40, 1), (128, 1)])
@pytest.mark.parametrize("name", ["cap", "all"])
def test_head_groups(dev, name, hq, hkv):
    check_varlen(dev, [70, 3, 150], hq, hkv, 64, lead=2, seed=11, **rule_for(name, [70, 3, 150], hq, dev))


@pytest.mark.parametrize("d", [16, 48, 80, 96, 112, 128])
@pytest.mark.parametrize("layout", ["head-major", "padded", "plain"])
@pytest.mark.parametrize("name", ["slopes", "all"])
def test_head_dims_and_layouts(dev, name, d, layout):
    check_varlen(dev, [140, 61], 6, 3, d, layout=layout, lead=1, tail=2, seed=20, **rule_for(name, [140, 61], 6, dev))


@pytest.mark.parametrize("name", list(RULES))
def test_padded_batch(dev, name):
    """Prefixes longer than what a sample uses, and samples of which nothing is used."""
    rule = rule_for(name, [200] * 4, 4, dev)
    check_varlen(dev, [200] * 4, 4, 2, 64, used=[200, 1, 0, 77], seed=30, **rule)
    rule = rule_for(name, [256] * 3, 8, dev, 2)
    check_varlen(dev, [256] * 3, 8, 2, 128, used=[129, 128, 255], seed=31, **rule)


@pytest.mark.parametrize("prefix", [1, 127, 128, 129, 300, 640, 900])
def test_prefixes_about_tiles(dev, prefix):
    check_varlen(dev, [900, 50], 4, 1, 64, prefix=[prefix, 0], seed=32)
    check_varlen(dev, [900], 4, 4, 128, prefix=[prefix], cap=10.0, seed=33)


@pytest.mark.parametrize("name", ["cap", "slopes", "prefix", "all"])
def test_long_and_many_samples(dev, name):
    check_varlen(dev, [2500, 700], 8, 2, 128, seed=40, **rule_for(name, [2500, 700], 8, dev))
    check_varlen(dev, [3, 1, 0, 8] * 120, 4, 4, 64, seed=41, **rule_for(name, [3, 1, 0, 8] * 120, 4, dev))


@pytest.mark.parametrize("cap", [0.25, 1.0, 50.0, 1000.0])
@pytest.mark.parametrize("qscale", [1e-3, 5.0, 40.0, 400.0])
def test_caps(dev, cap, qscale):
    """From scores far below the cap to all of them at it, forward; gradients where they are not
    below what bf16 holds."""
    check_varlen(dev, [260, 90], 4, 2, 64, cap=cap, seed=50, qscale=qscale, grads=qscale * 3 < 20 * cap)


@pytest.mark.parametrize("vscale", [1e-9, 1e9])
@pytest.mark.parametrize("towards", [1.0, -1.0])
def test_values_far_from_one_at_the_cap(dev, vscale, towards):
    """Scores all near the cap, or near its negative, and values far from 1, where the forward takes a
    fixed maximum (cap 55) and where it does not (56)."""
    m = pr()
    n, d = 400, 64
    q = torch.full((n, 2, d), 4.0, dtype=torch.bfloat16, device=dev)
    k = (towards * 4.0 + normal((n, 1, d), 53, dev).float() / 16).to(torch.bfloat16)
    v = (normal((n, 1, d), 54, dev).float() * vscale).to(torch.bfloat16)
    for cap in (55.0, 56.0):
        o, lse = m.attn_varlen_fwd(q, k, v, ints([0, n], dev), scale=0.125, score_cap=cap, return_lse=True)
        ref = sample_reference(q, k, v, 0.125, cap)
        assert_within(o, *ref["o"], "o")
        assert float((lse.double() - ref["lse"]).abs().max()) <= ref["rule"] + 2.0 ** -11 * (1 + float(ref["lse"].abs().max()))


@pytest.mark.parametrize("rule", [dict(score_cap=0.5), dict(score_cap=5.0), dict(score_cap=50.0), dict(score_cap=100.0),
                                  dict(score_cap=500.0), dict(slopes=True), dict(score_cap=30.0, slopes=True)], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_a_row_of_one_key_is_its_value(dev, rule, d):
    """The first row of a causal sample, to the bit: its weight and the sum it is divided by are the same."""
    m, g = pr(), torch.Generator("cuda").manual_seed(41)
    lengths = [1] * 150 + [2, 70, 300, 1, 513]
    n, hq, hkv = sum(lengths), 8, 2
    rule = dict(rule)
    if rule.pop("slopes", False):
        rule["distance_slopes"] = series(hq, dev)
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=dev)
    q, k, v = (torch.randn((n, h, d), generator=g, device=dev).bfloat16() for h in (hq, hkv, hkv))
    first = cu[:-1].long()
    for sharp in (0.1, 1.0, 6.0, 40.0):
        o = m.attn_varlen_fwd(q * sharp, k, v, cu, **rule)
        assert torch.equal(o[first], v[first].repeat_interleave(hq // hkv, dim=1))


@pytest.mark.parametrize("lengths,hq,hkv,d", [([1500], 8, 2, 128), ([130, 300, 900], 4, 4, 64), ([100, 128, 77], 4, 1, 80)], ids=str)
@pytest.mark.parametrize("cap,sloped", [(50.0, False), (20.0, False), (100.0, True), (200.0, False)])
def test_gradients_of_sharp_capped_scores(dev, lengths, hq, hkv, d, cap, sloped):
    """Rows that one key has nearly to itself: their D is nearly that key's dP, and the rounding of the
    output that comes in would show.  Off by the roundings of ds and of the result to bf16 alone: 2^-8 / sqrt(3)
    of a value's binade is 1.66e-3 of the values (mean square, mantissas spread evenly over their
    logarithm), both 2.35e-3; with 16e-6 cap from the tanh at most, 1.5e-3 of it on average for these
    caps, sqrt(2.35^2 + 1.5^2) = 2.8e-3."""
    m, g = pr(), torch.Generator("cuda").manual_seed(31)
    n = sum(lengths)
    q, k, v, dout = (torch.randn((n, h, d), generator=g, device=dev).bfloat16() for h in (hq, hkv, hkv, hq))
    q *= 6
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device=dev)
    slopes = series(hq, dev) if sloped else None
    o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True, score_cap=cap, distance_slopes=slopes)
    got = m.attn_varlen_bwd(dout, q, k, v, o, lse, cu, score_cap=cap, distance_slopes=slopes)
    refs = [sample_reference(*(x[a:b] for x in (q, k, v)), 1 / math.sqrt(d), cap, slopes, dout=dout[a:b])
            for a, b in zip(cu.tolist(), cu.tolist()[1:])]
    for i, name in enumerate(("dq", "dk")):
        want = torch.cat([r[name][0] for r in refs])
        err = float((got[i].double() - want).norm() / want.norm())
        assert err <= 2.8e-3, (name, err)


@pytest.mark.parametrize("cap,scale", [(1e-25, 1e-22), (1e-3, 1e3), (1e-12, 1e-16), (1e20, 1e16), (2e4, 0.125)])
def test_caps_and_scales_at_the_ends(dev, cap, scale):
    """Caps and scales whose powers leave binary32: scores moderate against the cap all the same."""
    spread = 0.6 * cap / scale / 64.0                        # |q.k| up to about 0.6 cap / scale
    m = pr()
    q, k = ((normal((90, 1, 64), 55 + i, dev).float() * (spread if i == 0 else 1.0)).to(torch.bfloat16) for i in range(2))
    v = normal((90, 1, 64), 57, dev)
    o = m.attn_varlen_fwd(q, k, v, ints([0, 90], dev), scale=scale, score_cap=cap)
    ref = sample_reference(q, k, v, scale, cap)
    if cap <= 2e4:                                           # (beyond, binary32 scores of that size mean little)
        assert_within(o, *ref["o"], "o")
    assert bool((o.double().abs() <= 1.01 * v.double().abs().max()).all())


def test_scores_of_any_size_with_slopes(dev):
    """Uncapped: however large the scores, the largest weight is 1 and one of the keys' values comes
    out, as they are too far apart for two."""
    m = pr()
    n = 300
    q, k, v = (normal((n, 2, 64), 58 + i, dev) for i in range(3))
    for size in (1e6, 1e15, 1e30):
        big = (k.float() * size).to(torch.bfloat16)
        for causal in (True, False):
            o = m.attn_varlen_fwd(q, big, v, ints([0, n], dev), causal=causal, distance_slopes=series(2, dev))
            s = torch.einsum("ihd,jhd->hij", q.double(), big.double())
            if causal:
                s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=dev).triu(1), -math.inf)
            best = s.argmax(dim=2)                           # [heads, rows]
            top2 = s.topk(2, dim=2).values
            # ahead by more than binary32's error in the scores, and than the bias can make up for
            ahead = top2[..., 0] - top2[..., 1]
            clear = (ahead > 1e-4 * top2[..., 0].abs()) & (0.125 * ahead > 0.5 * n + 50)
            want = torch.stack([v[best[h], h] for h in range(2)])
            got = o.transpose(0, 1)
            assert bool((got[clear] == want[clear]).all()) and not bool(o.isnan().any())


@pytest.mark.parametrize("size", [1e4, 1e8, 3e9, 1e10, 1e13, 1e30])
def test_large_scores_after_small_ones(dev, size):
    """Keys of ordinary scores, then one whose score is far larger: the rows that see it take its value."""
    m, n = pr(), 700
    q, k, v = (normal((n, 1, 64), 90 + i, dev) for i in range(3))
    for at in (600, 20):
        for d in (0, 8):                                     # of q and k: the large key's direction
            q[:, 0, d] = 1.0
            big = k.clone()
            big[at, 0] = 0.0
            big[at, 0, d] = size
            o = m.attn_varlen_fwd(q, big, v, ints([0, n], dev), distance_slopes=series(1, dev, 1e-3))
            assert bool((o[at:] == v[at]).all()) and not bool(o.isnan().any())
            ref = sample_reference(q[:at], big[:at], v[:at], 0.125, 0.0, series(1, dev, 1e-3))
            assert_within(o[:at], *ref["o"], "o")


@pytest.mark.parametrize("first", [0.0, -0.01, 0.02, 4.0, 40.0])
@pytest.mark.parametrize("causal", [True, False])
def test_slopes(dev, first, causal):
    """None, towards far keys, shallow, and so steep that a row sees its neighbours alone."""
    check_varlen(dev, [700, 130], 4, 4, 64, slopes=series(4, dev, first), causal=causal, seed=51)
    check_varlen(dev, [1500], 2, 1, 128, slopes=series(2, dev, first), causal=causal, seed=52)


def test_infinite_and_nan_scores(dev):
    """A score of +-infinity is capped; a NaN comes out in the rows that see it, and in no other."""
    m = pr()
    n, d = 300, 64
    q, k, v = (normal((n, 1, d), 60 + i, dev) for i in range(3))
    q[:, :, 0] = 1.0
    k[:, :, 0] = 0.0
    k[7, 0, 0], k[9, 0, 0] = 3e38, -3e38
    cu = ints([0, n], dev)
    o = m.attn_varlen_fwd(q, k, v, cu, scale=16.0, score_cap=5.0)
    capped = torch.tanh(16.0 * (q[:, 0].double() @ k[:, 0].double().t()) / 5.0) * 5.0
    capped = capped.masked_fill(torch.ones_like(capped, dtype=torch.bool).triu(1), -math.inf)
    p = capped.softmax(-1)
    x = v[:, 0].double()
    assert_within(o[:, 0], p @ x, U * (p @ x).abs() + (U + B32 + 16e-6 * 5.0) * (p @ x.abs()), "o")
    k[150, 0, 3] = float("nan")
    for rule in (dict(score_cap=5.0), dict(distance_slopes=series(1, dev)), dict(prefix_lens=ints([0], dev))):
        o, lse = m.attn_varlen_fwd(q, k, v, cu, scale=0.001, return_lse=True, **rule)
        assert not bool(o[:150].isnan().any()) and bool(o[150:].isnan().all()) and bool(lse[0, 150:].isnan().all())


def test_no_prefix_is_the_plain_operator(dev):
    m = pr()
    q, k, v = qkv_views(700, 8, 2, 128, 61, dev, "fused")
    cu = ints([0, 300, 700], dev)
    want, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True)
    got, lse2 = m.attn_varlen_fwd(q, k, v, cu, return_lse=True, prefix_lens=ints([0, -3], dev))
    assert torch.equal(want, got) and torch.equal(lse, lse2)
    dout = normal(q.shape, 62, dev)
    for a, b in zip(m.attn_varlen_bwd(dout, q, k, v, want, lse, cu),
                    m.attn_varlen_bwd(dout, q, k, v, got, lse2, cu, prefix_lens=ints([0, 0], dev))):
        assert torch.equal(a, b)


def test_autograd(dev):
    """Leaves with shared heads, broadcast gradients and a head-major layout."""
    m = pr()
    q, k, v = (normal((90, h, 64), 63 + h, dev).requires_grad_() for h in (4, 2, 1))
    kk, vv = k, v.expand(90, 2, 64)
    slopes, prefix, cu = series(4, dev), ints([10, 0], dev), ints([0, 40, 90], dev)
    o = m.apply_attn(q, kk, vv, cu, score_cap=4.0, distance_slopes=slopes, prefix_lens=prefix)
    g = normal((1, 4, 64), 70, dev).expand(90, 4, 64)
    o.backward(g)
    for a, b, pre in ((0, 40, 10), (40, 90, 0)):
        ref = sample_reference(q[a:b], kk[a:b], vv[a:b], 0.125, 4.0, slopes, pre, True, g[a:b])
        assert_within(o[a:b], *ref["o"], "o")
        assert_within(q.grad[a:b], *ref["dq"], "dq")
        assert_within(k.grad[a:b], *ref["dk"], "dk")
        dv, tol = (x.sum(dim=1, keepdim=True) for x in ref["dv"])          # the heads' gradients, added in bf16
        assert_within(v.grad[a:b], dv, tol + 2.0 ** -8 * dv.abs(), "dv")


def check_paged(dev, new, kv, page, hq, hkv, d, cap=0.0, slopes=None, prefix=None, causal=True, seed=1, max_kv_len=0,
                qscale=1.5, extra_pages=0):
    m = pr()
    cache, table, k_of, v_of = make_paged(dev, kv, page, hkv, d, seed)
    cu_list = offsets(new)
    q = normal((cu_list[-1], hq, d), seed + 5, dev) * qscale
    if extra_pages:                                          # a table wider than the sequences: more splits
        table = torch.cat([table, torch.full((len(kv), extra_pages), 1 << 30, dtype=torch.int32, device=dev)], dim=1)
    o = m.attn_paged(q, cache, table, ints(kv, dev), ints(cu_list, dev), causal=causal, max_kv_len=max_kv_len, score_cap=cap,
                     distance_slopes=slopes, prefix_lens=None if prefix is None else ints(prefix, dev))
    torch.cuda.synchronize()
    for i, (a, n) in enumerate(zip(cu_list, new)):
        if n == 0:
            continue
        ref = sample_reference(q[a:a + n], k_of[i], v_of[i], 1 / math.sqrt(d), cap, slopes,
                               None if prefix is None else min(prefix[i], kv[i]), causal)
        assert_within(o[a:a + n], *ref["o"], "rows %d..%d" % (a, a + n))
    assert not m.attn_fault()


@pytest.mark.parametrize("name", list(RULES))
@pytest.mark.parametrize("page", [8, 24, 64])
def test_paged(dev, name, page):
    """One token each, a few, chunks; sequences of a single token, and of whole pages."""
    for new, kv, heads, d in (([1] * 5, [1, 7, 64, 500, 1025], (8, 2), 128), ([3, 1, 0, 7], [3, 200, 9, 640], (4, 4), 64),
                              ([150, 1, 300], [400, 90, 300], (6, 2), 80), ([1, 1], [3000, 1], (1, 1), 64)):
        rule = rule_for(name, kv, heads[0], dev, page)
        check_paged(dev, new, kv, page, *heads, d, seed=page, **rule)


@pytest.mark.parametrize("name", ["cap", "slopes", "all"])
def test_paged_splits(dev, name):
    """Long caches of few rows: clusters, splits and their join, in both kernels."""
    for new, kv, heads, d in (([1], [20000], (2, 1), 128), ([1, 1], [9000, 40], (8, 1), 64), ([40], [20000], (4, 2), 128),
                              ([300], [12000], (1, 1), 64)):
        rule = rule_for(name, kv, heads[0], dev)
        check_paged(dev, new, kv, 64, *heads, d, seed=7, **rule)
        check_paged(dev, new, kv, 64, *heads, d, seed=8, max_kv_len=max(kv), extra_pages=700, **rule)


def test_paged_steep_slopes_and_both_directions(dev):
    for first in (4.0, -0.02, 40.0):
        check_paged(dev, [1, 5], [3000, 700], 32, 4, 4, 64, slopes=series(4, dev, first), seed=9)
        check_paged(dev, [200], [3000], 32, 4, 4, 64, slopes=series(4, dev, first), seed=10)
    check_paged(dev, [3, 200], [700, 900], 32, 4, 2, 64, slopes=series(4, dev), cap=9.0, causal=False, seed=11)


def test_paged_nan_in_a_key_comes_out(dev):
    m = pr()
    cache, table, k_of, v_of = make_paged(dev, [500], 64, 1, 64, 12)
    cache.k_pages[table[0, 3], 5, 0, 9] = float("nan")       # key 197
    for rows in (1, 400):
        q = normal((rows, 2, 64), 13, dev)
        for rule in (dict(score_cap=5.0), dict(distance_slopes=series(2, dev)), dict(prefix_lens=ints([300], dev)),
                     dict(prefix_lens=ints([190], dev))):
            o = m.attn_paged(q, cache, table, ints([500], dev), ints([0, rows], dev), **rule)
            first = 0 if rule.get("prefix_lens") is not None and int(rule["prefix_lens"]) > 197 else max(0, 197 - (500 - rows))
            assert bool(o[first:].isnan().all()) and not bool(o[:first].isnan().any())


def test_graph_and_streams(dev):
    """Captured with the rule's arrays, replayed on other values of them; and on another stream."""
    m = pr()
    q, k, v = qkv_views(600, 4, 2, 64, 80, dev, "fused")
    dout, cu = normal((600, 4, 64), 81, dev), ints([0, 200, 600], dev)
    slopes, prefix = series(4, dev), ints([0, 0], dev)
    rule = dict(score_cap=6.0, distance_slopes=slopes, prefix_lens=prefix)

    def train(stream=None):
        o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True, stream=stream, **rule)
        return (o, *m.attn_varlen_bwd(dout, q, k, v, o, lse, cu, stream=stream, **rule))

    train()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train()
    for pre, first in (([50, 399], 0.25), ([200, 1], 2.0)):
        prefix.copy_(ints(pre, dev))
        slopes.copy_(series(4, dev, first))
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(((0, 200), (200, 600))):
            ref = sample_reference(q[a:b], k[a:b], v[a:b], 0.125, 6.0, slopes, pre[i], True, dout[a:b])
            for x, name in zip(got, ("o", "dq", "dk", "dv")):
                assert_within(x[a:b], *ref[name], name)
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    other = train(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, other))


def test_refusals(dev):
    m = pr()
    q, k, v = qkv_views(20, 4, 2, 64, 90, dev, "plain")
    cu = ints([0, 20], dev)
    good = series(4, dev)
    for bad in (dict(distance_slopes=good[:2]), dict(distance_slopes=good.double()), dict(distance_slopes=good.cpu()),
                dict(distance_slopes=good.repeat(2)[::2]), dict(prefix_lens=ints([1, 2], dev)),
                dict(prefix_lens=ints([1], dev, torch.int64)), dict(prefix_lens=ints([1], torch.device("cpu"))),
                dict(distance_slopes=good.clone().requires_grad_())):
        with pytest.raises(ValueError):
            m.attn_varlen_fwd(q, k, v, cu, **bad)
    for bad in (dict(score_cap=-1.0), dict(score_cap=float("nan")), dict(score_cap=float("inf")),
                dict(prefix_lens=ints([1], dev), causal=False)):
        with pytest.raises(m.RopeError):
            m.attn_varlen_fwd(q, k, v, cu, **bad)
