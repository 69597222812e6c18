"""NaN and scores past binary32's range in queries and keys that rows do see (needs a GB300): they
reach the rows' results however the keys are split, and no other row's."""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import assert_within, causal_mask, normal, sample_reference  # noqa: E402
from test_gpu_attention import make_paged  # noqa: E402


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


def check_rows(o, spoiled, ref, what):
    """Rows (token, head) of ``spoiled`` are NaN throughout, the others within the bound."""
    assert bool(o[spoiled].isnan().all()), what
    assert_within(o[~spoiled], ref[0][~spoiled], ref[1][~spoiled], what)


@pytest.mark.parametrize("new,d", [(1, 64), (1, 128), (3, 128), (40, 64), (40, 128)])
def test_paged_nan_and_overflow_split_or_not(dev, new, d):
    """One call under two plans: split over a second launch, and (a bound of 16 keys) not."""
    m = pr()
    kv, hq, hkv, page, at = 20000, 4, 2, 64, 7000
    cu = torch.tensor([0, new], dtype=torch.int32, device=dev)
    lens = torch.tensor([kv], dtype=torch.int32, device=dev)
    seen = causal_mask(new, kv, True, dev)
    for spoil in ("query", "key", "overflow", "below"):
        cache, table, ks, vs = make_paged(dev, [kv], page, hkv, d, 40)
        q = normal((new, hq, d), 41, dev)
        pages, slot = cache.k_pages, (int(table[0, at // page]), at % page)
        spoiled = torch.zeros((new, hq), dtype=torch.bool, device=dev)
        if spoil in ("overflow", "below"):     # column 0 matters to one row and one key alone
            ks[0][:, 1, 0], pages[:, :, 1, 0], q[:, 2:, 0] = 0, 0, 0
        ref = sample_reference(q, ks[0], vs[0], 1 / math.sqrt(d), seen)["o"]
        if spoil == "query":
            q[new - 1, 1, 5] = float("nan")
            spoiled[new - 1, 1] = True
        elif spoil == "key":
            pages[slot][1, 3] = float("nan")
            spoiled[:, 2:] = True
        elif spoil == "overflow":
            q[new - 1, 3, 0], pages[slot][1, 0] = 2.0 ** 70, 2.0 ** 70
            spoiled[new - 1, 3] = True
        else:                                   # a score of -infinity: the key has no weight
            q[new - 1, 3, 0], pages[slot][1, 0] = 2.0 ** 70, -2.0 ** 70
            without = seen.clone()
            without[:, at] = False
            less = sample_reference(q, ks[0], vs[0], 1 / math.sqrt(d), without)["o"]
            for x, y in zip(ref, less):
                x[new - 1, 3] = y[new - 1, 3]
        for bound in (0, 16):
            need = m.attn_paged_workspace_bytes(q, cache, table, lens, cu, max_kv_len=bound)
            assert (need > 0) == (bound == 0)
            o = m.attn_paged(q, cache, table, lens, cu, max_kv_len=bound)
            check_rows(o, spoiled, ref, "%s, %d bytes of workspace" % (spoil, need))


@pytest.mark.parametrize("d", [64, 128])
def test_packed_nan_query(dev, d):
    """Out and lse of the row are NaN (lse is not that of a row without keys); no other row's."""
    m = pr()
    n, hq, hkv = 300, 4, 2
    q, k, v = normal((n, hq, d), 50, dev), normal((n, hkv, d), 51, dev), normal((n, hkv, d), 52, dev)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    ref = sample_reference(q, k, v, 1 / math.sqrt(d), causal_mask(n, n, True, dev))
    spoiled = torch.zeros((n, hq), dtype=torch.bool, device=dev)
    for row, head in ((0, 1), (130, 2), (299, 3)):
        q[row, head, 7] = float("nan")
        spoiled[row, head] = True
    o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True)
    check_rows(o, spoiled, ref["o"], "o")
    assert bool(lse.t()[spoiled].isnan().all())
    err = (lse.double() - ref["lse"]).abs().t()[~spoiled]
    assert float(err.max()) <= 2.0 ** -11 * (1 + float(ref["lse"].abs().max()))


@pytest.mark.parametrize("level", [0.0, 2.0 ** 10, -2.0 ** 12, 2.0 ** 14])
@pytest.mark.parametrize("n,causal", [(100, True), (300, False)])
def test_gradients_of_large_scores(dev, level, n, causal):
    """Scores level + x with x of a few units, exact in binary32: what the backward loses is its
    exponent's rounding against lse, at most |lse| 2^-22 of a weight (lse's own two roundings, that
    of lse log2(e) and that of scale log2(e), 2^-24 of |lse| each)."""
    m = pr()
    d = 64
    q, k = torch.zeros((n, 1, d), device=dev), torch.zeros((n, 1, d), device=dev)
    gen = torch.Generator(device=dev).manual_seed(60)
    q[..., :2], k[..., 0] = 1.0, level
    k[..., 1] = torch.randint(-64, 65, (n, 1), generator=gen, device=dev) / 32
    q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
    v, dout = normal((n, 1, d), 61, dev), normal((n, 1, d), 62, dev)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    seen = causal_mask(n, n, causal, dev)
    ref = sample_reference(q, k, v, 1.0, seen, dout)
    o, lse = m.attn_varlen_fwd(q, k, v, cu, causal=causal, scale=1.0, return_lse=True)
    got = m.attn_varlen_bwd(dout, q, k, v, o, lse, cu, causal=causal, scale=1.0)
    rel = float(ref["lse"].abs().max()) * 2.0 ** -22
    Q, K, V, G = (x[:, 0].double() for x in (q, k, v, dout))
    p = torch.where(seen, torch.exp(Q @ K.t() - ref["lse"][0][:, None]), 0.0)
    dP, D = G @ V.t(), (G * (p @ V)).sum(1, keepdim=True)
    ds = p * (dP.abs() + 2 * D.abs())              # a row's weights are off by one factor, and D with them
    assert_within(o, *ref["o"], "o")
    assert float((lse.double() - ref["lse"]).abs().max()) <= float(ref["lse"].abs().max()) * 2.0 ** -23 + 2.0 ** -18
    for x, name, more in zip(got, ("dq", "dk", "dv"), (ds @ K.abs(), ds.t() @ Q.abs(), p.t() @ G.abs())):
        value, bound = ref[name]
        assert_within(x, value, bound + rel * more[:, None], name)
