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
