"""Packed and paged attention against the binary64 definition (needs a GB300): forward,
gradients, layouts, masks that leave rows empty, garbage in places no row may read."""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import assert_within, causal_mask, normal, offsets, sample_reference  # noqa: E402


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


def qkv_views(T, hq, hkv, d, seed, dev, layout):
    """q, k, v with the given memory layout."""
    if layout == "fused":
        x = normal((T, hq + 2 * hkv, d), seed, dev)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if layout == "head-major":
        return tuple(normal((h, T, d), seed + i, dev).transpose(0, 1) for i, h in enumerate((hq, hkv, hkv)))
    if layout == "padded":       # strides that are no multiple of one another
        return tuple(normal((T, h, d + 8), seed + i, dev)[:, :, :d] for i, h in enumerate((hq, hkv, hkv)))
    return tuple(normal((T, h, d), seed + i, dev) for i, h in enumerate((hq, hkv, hkv)))


def check_varlen(dev, lengths, hq, hkv, d, causal, layout="fused", used=None, lead=0, tail=0, seed=1, scale=None,
                 grads=True, poison=True, qscale=1.5):
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
    if poison:
        for x in (q, k, v, dout):
            x[~inside] = float("nan")
    cu = torch.tensor(cu_list, dtype=torch.int32, device=dev)
    su = torch.tensor(used, dtype=torch.int32, device=dev) if used != list(lengths) else None
    o, lse = m.attn_varlen_fwd(q, k, v, cu, causal=causal, scale=scale, seq_used=su, return_lse=True)
    o_only = m.attn_varlen_fwd(q, k, v, cu, causal=causal, scale=scale, seq_used=su)
    got = {"o": o}
    if grads:
        got.update(zip(("dq", "dk", "dv"), m.attn_varlen_bwd(dout, q, k, v, o, lse, cu, causal=causal, scale=scale,
                                                             seq_used=su)))
    torch.cuda.synchronize()
    assert torch.equal(o, o_only)
    sc = 1 / math.sqrt(d) if scale is None else scale
    for a, n in zip(cu_list, used):
        if n == 0:
            continue
        ref = sample_reference(q[a:a + n], k[a:a + n], v[a:a + n], sc, causal_mask(n, n, causal, dev),
                               dout[a:a + n] if grads else None)
        for name, x in got.items():
            assert_within(x[a:a + n], *ref[name], "%s of rows %d..%d" % (name, a, a + n))
        err = (lse[:, a:a + n].double() - ref["lse"]).abs()
        assert float(err.max()) <= 2.0 ** -11 * (1 + float(ref["lse"].abs().max()))
    for name, x in got.items():
        assert not bool(x[~inside].any()), name + " of rows outside is not zero"
    assert bool((lse[:, ~inside] == -math.inf).all())
    assert not m.attn_fault()


LENGTHS = [[1], [2, 0, 1], [5, 17, 33, 9], [64, 64], [127, 1, 128, 129], [300, 0, 0, 255, 1], [513], [1000, 37]]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_lengths(dev, lengths, causal):
    check_varlen(dev, lengths, 4, 2, 64, causal, lead=3, tail=5)
    check_varlen(dev, lengths, 8, 2, 128, causal, lead=0, tail=0, seed=3)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (6, 2), (5, 1), (14, 2), (8, 1), (16, 1), (40, 1), (128, 1), (66, 1)])
def test_head_groups(dev, hq, hkv):
    check_varlen(dev, [70, 3, 150], hq, hkv, 64, True, lead=2, seed=11)
    check_varlen(dev, [131], hq, hkv, 128, False, seed=12)


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("layout", ["fused", "head-major", "padded", "plain"])
def test_head_dims_and_layouts(dev, d, layout):
    check_varlen(dev, [140, 61], 6, 3, d, True, layout, lead=1, tail=2, seed=20)


@pytest.mark.parametrize("causal", [True, False])
def test_padded_batch(dev, causal):
    check_varlen(dev, [200, 200, 200, 200], 4, 2, 64, causal, used=[200, 1, 0, 77], seed=30)
    check_varlen(dev, [256] * 3, 8, 2, 128, causal, used=[129, 128, 255], seed=31)


def test_long_sample_and_many_samples(dev):
    check_varlen(dev, [2500, 700], 8, 2, 128, True, seed=40)
    check_varlen(dev, [3, 1, 0, 8] * 120, 4, 4, 64, True, seed=41)
    check_varlen(dev, [1900], 4, 1, 64, False, seed=42)


@pytest.mark.parametrize("qscale", [1e-3, 20.0, 200.0])
def test_score_ranges(dev, qscale):
    """Scores near zero, and so large that one key takes nearly all the weight."""
    check_varlen(dev, [260, 90], 4, 2, 64, True, seed=50, qscale=qscale, grads=qscale < 100)


def test_rising_maximum(dev):
    """Scores that grow along the keys, so that every tile raises the running maximum."""
    m = pr()
    n, d = 900, 64
    q = torch.ones((n, 2, d), dtype=torch.bfloat16, device=dev)
    k = (torch.arange(n, device=dev).float()[:, None, None] / 16).expand(n, 1, d).to(torch.bfloat16)
    v = normal((n, 1, d), 60, dev)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    for causal in (True, False):
        for kk in (k, k.flip(0).contiguous()):
            o = m.attn_varlen_fwd(q, kk, v, cu, causal=causal, scale=0.125)
            ref = sample_reference(q, kk, v, 0.125, causal_mask(n, n, causal, dev))
            assert_within(o, *ref["o"], "o")


def test_scores_of_the_lowest_value(dev):
    """Products near binary32's lowest finite scores: every weight stays defined."""
    m = pr()
    n, d = 200, 64
    q = torch.full((n, 1, d), -2.0 ** 60, dtype=torch.bfloat16, device=dev)
    k = torch.full((n, 1, d), 2.0 ** 60, dtype=torch.bfloat16, device=dev)
    v = normal((n, 1, d), 61, dev)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    o = m.attn_varlen_fwd(q, k, v, cu, scale=1.0)          # all scores equal: -2^126
    w = torch.arange(1, n + 1, device=dev, dtype=torch.float64)[:, None, None]
    ref = v.double().cumsum(dim=0) / w
    tol = 2 * 2.0 ** -8 * (v.double().abs().cumsum(dim=0) / w + ref.abs()) + 1e-30
    assert_within(o, ref, tol, "o")


def test_repeats_bit_for_bit(dev):
    m = pr()
    q, k, v = qkv_views(1500, 8, 2, 128, 70, dev, "fused")
    cu = torch.tensor([0, 400, 401, 1500], dtype=torch.int32, device=dev)
    dout = normal((1500, 8, 128), 71, dev)
    first = None
    for _ in range(3):
        o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True)
        now = (o, lse, *m.attn_varlen_bwd(dout, q, k, v, o, lse, cu))
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def test_gradient_against_differences(dev):
    """The directional derivative of sum(dout * o), in binary64 from the plain forward,
    equals the kernel's gradient along that direction within the gradient's own bound."""
    m = pr()
    lengths, hq, hkv, d = [50, 81], 4, 2, 64
    q, k, v = qkv_views(sum(lengths), hq, hkv, d, 80, dev, "plain")
    dout = normal(q.shape, 84, dev)
    cu_list = offsets(lengths)
    cu = torch.tensor(cu_list, dtype=torch.int32, device=dev)
    o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True)
    got = m.attn_varlen_bwd(dout, q, k, v, o, lse, cu)
    sc = 1 / math.sqrt(d)

    def value(xs):
        total = 0.0
        for a, b in zip(cu_list, cu_list[1:]):
            ref = sample_reference(*(x[a:b] for x in xs), sc, causal_mask(b - a, b - a, True, dev))
            total += float((ref["o"][0] * dout[a:b].double()).sum())
        return total

    bounds = [torch.zeros(x.shape, dtype=torch.float64, device=dev) for x in (q, k, v)]
    for a, b in zip(cu_list, cu_list[1:]):
        ref = sample_reference(q[a:b], k[a:b], v[a:b], sc, causal_mask(b - a, b - a, True, dev), dout[a:b])
        for t, name in zip(bounds, ("dq", "dk", "dv")):
            t[a:b] = ref[name][1]
    for which in range(3):
        direction = torch.randn(got[which].shape, dtype=torch.float64, device=dev,
                                generator=torch.Generator(device=dev).manual_seed(90 + which))
        h = 1e-4
        plus, minus = ([x.double() + (s * h * direction if i == which else 0) for i, x in enumerate((q, k, v))]
                       for s in (1, -1))
        slope = (value(plus) - value(minus)) / (2 * h)
        mine = float((got[which].double() * direction).sum())
        # the third-order remainder of the difference is below 1e-5 of the terms
        room = float((bounds[which] * direction.abs()).sum()) + 1e-5 * float((got[which].double() * direction).abs().sum())
        assert abs(slope - mine) <= room


def test_autograd_and_broadcast(dev):
    """apply_attn against autograd through the binary64 definition, with a value tensor
    broadcast over its heads and a broadcast output gradient."""
    m = pr()
    n, hq, hkv, d = 90, 4, 2, 64
    q, k = normal((n, hq, d), 91, dev).requires_grad_(), normal((n, hkv, d), 92, dev).requires_grad_()
    v1 = normal((n, 1, d), 93, dev).requires_grad_()
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    o = m.apply_attn(q, k, v1.expand(n, hkv, d), cu)
    g = normal((1, 1, d), 94, dev)
    o.backward(g.expand(n, hq, d))
    ref = sample_reference(q.detach(), k.detach(), v1.detach().expand(n, hkv, d), 1 / math.sqrt(d),
                           causal_mask(n, n, True, dev), g.expand(n, hq, d))
    assert_within(o.detach(), *ref["o"], "o")
    assert_within(q.grad, *ref["dq"], "dq")
    assert_within(k.grad, *ref["dk"], "dk")
    x, t = ref["dv"]
    # the sum over heads is rounded to bf16 once more
    x = x.sum(dim=1, keepdim=True)
    assert_within(v1.grad, x, t.sum(dim=1, keepdim=True) + 2.0 ** -8 * x.abs() * 1.01, "dv")


def test_other_stream(dev):
    """The explicit stream, with temporaries the call allocates itself."""
    m = pr()
    q, k, v = qkv_views(600, 4, 2, 64, 95, dev, "fused")
    cu = torch.tensor([0, 600], dtype=torch.int32, device=dev)
    dout = normal((600, 4, 64), 96, dev)
    o0, lse0 = m.attn_varlen_fwd(q, k, v, cu, return_lse=True)
    g0 = m.attn_varlen_bwd(dout, q, k, v, o0, lse0, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o1, lse1 = m.attn_varlen_fwd(q, k, v, cu, return_lse=True, stream=s)
    g1 = m.attn_varlen_bwd(dout, q, k, v, o1, lse1, cu, stream=s)
    junk = torch.full((600 * 4,), 7.0, device=dev)          # would reuse a freed workspace
    s.synchronize()
    assert torch.equal(o0, o1) and all(torch.equal(a, b) for a, b in zip(g0, g1)) and float(junk[0]) == 7.0


def test_graph_capture(dev):
    m = pr()
    q, k, v = qkv_views(300, 4, 2, 64, 97, dev, "fused")
    cu = torch.tensor([0, 100, 300], dtype=torch.int32, device=dev)
    dout = normal((300, 4, 64), 98, dev)

    def step():
        o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True)
        return (o, *m.attn_varlen_bwd(dout, q, k, v, o, lse, cu))

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    q.copy_(normal(q.shape, 99, dev))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_invalid_offsets_stay_inside(dev):
    """cu_seqlens that decrease, run past the end or start below zero: no read or write
    outside the buffers (guard rows around the outputs stay as they were)."""
    m = pr()
    T = 200
    q, k, v = qkv_views(T, 4, 2, 64, 101, dev, "fused")
    for cu_list in ([0, 150, 90, 200], [-40, 60, 120], [0, 90, 5000], [300, 400, 500]):
        cu = torch.tensor(cu_list, dtype=torch.int32, device=dev)
        guard = torch.full((T + 2, 4, 64), 3.0, dtype=torch.bfloat16, device=dev)
        _, lse = m.attn_varlen_fwd(q, k, v, cu, out=guard[1:T + 1], return_lse=True)
        g = m.attn_varlen_bwd(q, q, k, v, guard[1:T + 1], lse, cu)
        torch.cuda.synchronize()
        assert bool((guard[0] == 3).all()) and bool((guard[T + 1] == 3).all()) and len(g) == 3
        assert not m.attn_fault()


# ---------------------------------------------------------------------------- paged

def make_paged(dev, kv, page, hkv, d, seed, layout="plain", width=None, fill=float("nan")):
    """Random keys and values of every sequence [kv_s, hkv, d], the cache that holds them
    with ``fill`` everywhere else, and the page table."""
    m = pr()
    need = [-(-max(n, 0) // page) for n in kv]
    n_pages = sum(need) + 3
    if layout == "heads-first":
        kp, vp = (torch.full((n_pages, hkv, page, d), fill, dtype=torch.bfloat16, device=dev).transpose(1, 2)
                  for _ in range(2))
    elif layout == "one-pool":
        pool = torch.full((n_pages, 2, page, hkv, d), fill, dtype=torch.bfloat16, device=dev)
        kp, vp = pool[:, 0], pool[:, 1]
    else:
        kp, vp = (torch.full((n_pages, page, hkv, d), fill, dtype=torch.bfloat16, device=dev) for _ in range(2))
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(need + [1]) if width is None else width
    table = torch.full((len(kv), width), -7, dtype=torch.int32)
    ks, vs = [], []
    for s, n in enumerate(kv):
        k, v = normal((max(n, 0), hkv, d), seed + 100 + s, dev), normal((max(n, 0), hkv, d), seed + 200 + s, dev)
        for i in range(need[s]):
            at = order.pop()
            table[s, i] = at
            rows = slice(i * page, min((i + 1) * page, n))
            kp[at, :rows.stop - rows.start], vp[at, :rows.stop - rows.start] = k[rows], v[rows]
        ks.append(k)
        vs.append(v)
    return m.PagedKVCache(kp, vp), table.to(dev), ks, vs


def check_paged(dev, new, kv, page, hq, hkv, d, causal=True, seed=1, layout="plain", width=None, max_kv_len=0, lead=0,
                tail=0):
    m = pr()
    cache, table, ks, vs = make_paged(dev, kv, page, hkv, d, seed, layout, width)
    cu_list = offsets(new, lead)
    T = cu_list[-1] + tail
    q = normal((T, hq, d), seed + 1, dev, 1.5)
    cu = torch.tensor(cu_list, dtype=torch.int32, device=dev)
    lens = torch.tensor(kv, dtype=torch.int32, device=dev)
    o = m.attn_paged(q, cache, table, lens, cu, causal=causal, max_kv_len=max_kv_len)
    torch.cuda.synchronize()
    inside = torch.zeros(T, dtype=torch.bool, device=dev)
    for s, (a, n) in enumerate(zip(cu_list, new)):
        inside[a:a + n] = True
        if n == 0:
            continue
        seen = causal_mask(n, ks[s].shape[0], causal, dev)
        pos = torch.arange(n, device=dev) + kv[s] - n
        seen = seen & (pos >= 0)[:, None]
        ref = sample_reference(q[a:a + n], ks[s], vs[s], 1 / math.sqrt(d), seen)
        assert_within(o[a:a + n], *ref["o"], "o of sequence %d" % s)
    assert not bool(o[~inside].any())
    assert not m.attn_fault()


@pytest.mark.parametrize("page", [8, 16, 24, 64, 128, 256])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 8, 2), (80, 5, 1)])
def test_paged_decode(dev, page, d, hq, hkv):
    check_paged(dev, [1, 1, 1, 1, 1], [1, 7, 130, 700, 64], page, hq, hkv, d, seed=5)


@pytest.mark.parametrize("page", [8, 24, 64, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_paged_chunks(dev, page, causal):
    check_paged(dev, [5, 0, 300, 1, 33], [9, 40, 300, 500, 1000], page, 8, 2, 128, causal, seed=6, lead=2, tail=3)
    check_paged(dev, [130, 3], [800, 3], page, 6, 2, 64, causal, seed=7)


@pytest.mark.parametrize("layout", ["plain", "heads-first", "one-pool"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (24, 2), (40, 1), (12, 4)])
def test_paged_layouts_and_groups(dev, layout, hq, hkv):
    check_paged(dev, [1, 2, 6], [333, 90, 6], 16, hq, hkv, 64, seed=8, layout=layout)
    check_paged(dev, [40, 1], [333, 900], 32, hq, hkv, 128, seed=9, layout=layout)


def test_paged_rows_that_see_nothing(dev):
    """Sequences with no key, fewer keys than new tokens, negative lengths."""
    check_paged(dev, [1, 3, 4], [0, 1, 4], 16, 4, 2, 64, seed=10)
    check_paged(dev, [3, 1, 20], [-5, 1, 2], 16, 4, 2, 128, seed=11)
    check_paged(dev, [3, 1, 20], [0, 0, 0], 16, 4, 2, 128, causal=False, seed=11)


@pytest.mark.parametrize("n", [1, 2, 30, 200])
def test_paged_batches_and_wide_tables(dev, n):
    """Page tables much wider than the lengths, with and without a bound on the lengths."""
    kv = [1 + (37 * i) % 411 for i in range(n)]
    for bound in (0, 411):
        check_paged(dev, [1] * n, kv, 16, 8, 2, 64, seed=12, width=500, max_kv_len=bound)
    check_paged(dev, [1] * n, kv, 16, 8, 2, 64, seed=12, max_kv_len=5)      # too low a bound: no key is cut off


def test_paged_long_cache(dev):
    check_paged(dev, [1, 2], [20011, 9000], 64, 8, 1, 128, seed=13)
    check_paged(dev, [1], [33000], 256, 4, 4, 64, seed=14)
    check_paged(dev, [140], [12345], 64, 8, 2, 128, seed=15)


def test_paged_invalid_page_ids(dev):
    """Page ids outside the pool read as zero keys and values."""
    m = pr()
    for new in (1, 50):
        cache, table, ks, vs = make_paged(dev, [200], 16, 2, 64, 16)
        table[0, 3], table[0, 7] = -1, cache.n_pages
        for x in (ks[0], vs[0]):
            x[48:64], x[112:128] = 0, 0
        q = normal((new, 4, 64), 17, dev)
        cu = torch.tensor([0, new], dtype=torch.int32, device=dev)
        o = m.attn_paged(q, cache, table, torch.tensor([200], dtype=torch.int32, device=dev), cu)
        ref = sample_reference(q, ks[0], vs[0], 0.125, causal_mask(new, 200, True, dev))
        assert_within(o, *ref["o"], "o")


def test_paged_past_the_table(dev):
    """kv_lens beyond the page table's width: keys past it are not read."""
    m = pr()
    cache, table, ks, vs = make_paged(dev, [160], 16, 2, 64, 18)
    q = normal((2, 4, 64), 19, dev)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    lens = torch.tensor([100000, 160], dtype=torch.int32, device=dev)
    o = m.attn_paged(q, cache, table.expand(2, -1).contiguous(), lens, cu)
    ref = sample_reference(q, ks[0], vs[0], 0.125, torch.ones((2, 160), dtype=torch.bool, device=dev))
    assert_within(o, *ref["o"], "o")


def test_paged_offsets_past_32_bits(dev):
    """A pool of more than 2^31 elements: pages at its far end."""
    m = pr()
    page, hkv, d = 256, 8, 128
    n_pages = (1 << 31) // (page * hkv * d) + 40
    kp = torch.empty((n_pages, page, hkv, d), dtype=torch.bfloat16, device=dev)
    vp = torch.empty_like(kp)
    kv = 1000
    k, v = normal((kv, hkv, d), 20, dev), normal((kv, hkv, d), 21, dev)
    far = [n_pages - 1, n_pages - 9, 2, n_pages - 30]
    for i, at in enumerate(far):
        n = min(page, kv - i * page)
        kp[at, :n], vp[at, :n] = k[i * page:i * page + n], v[i * page:i * page + n]
    cache = m.PagedKVCache(kp, vp)
    table = torch.tensor([far], dtype=torch.int32, device=dev)
    for new in (1, 60):
        q = normal((new, 16, d), 22, dev)
        cu = torch.tensor([0, new], dtype=torch.int32, device=dev)
        o = m.attn_paged(q, cache, table, torch.tensor([kv], dtype=torch.int32, device=dev), cu)
        ref = sample_reference(q, k, v, 1 / math.sqrt(d), causal_mask(new, kv, True, dev))
        assert_within(o, *ref["o"], "o")


def test_paged_workspace_and_stream(dev):
    m = pr()
    cache, table, ks, vs = make_paged(dev, [3000, 100], 64, 2, 128, 23)
    q = normal((2, 8, 128), 24, dev)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    lens = torch.tensor([3000, 100], dtype=torch.int32, device=dev)
    o = m.attn_paged(q, cache, table, lens, cu)
    need = m.attn_paged_workspace_bytes(q, cache, table, lens, cu)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=dev)     # NaN patterns
    assert torch.equal(o, m.attn_paged(q, cache, table, lens, cu, workspace=ws))
    if need:
        with pytest.raises(m.RopeError):
            m.attn_paged(q, cache, table, lens, cu, workspace=ws[:need - 1])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2 = m.attn_paged(q, cache, table, lens, cu, stream=s)
    junk = torch.full((max(need, 16) // 4 + 1,), 7.0, device=dev)
    s.synchronize()
    assert torch.equal(o, o2) and float(junk[0]) == 7.0


def test_refusals(dev):
    """What the binding refuses before the library sees it, and what the library refuses."""
    m = pr()
    x = normal((8, 8, 64), 1, dev)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    cu = torch.tensor([0, 8], dtype=torch.int32, device=dev)
    o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True)
    for args, kw in (((q.float(), k, v, cu), {}), ((q, k[:4], v, cu), {}), ((q, k, x[:, 5:], cu), {}),
                     ((q, k, v, cu.long()), {}), ((q, k, v, cu.cpu()), {}), ((q, k, v, cu), dict(out=o[:4])),
                     ((q, k, v, cu), dict(seq_used=torch.zeros(2, dtype=torch.int32, device=dev))),
                     ((q.transpose(1, 2), k, v, cu), {})):
        with pytest.raises(ValueError):
            m.attn_varlen_fwd(*args, **kw)
    for args in ((q, q, k, v, o, None, cu), (q[:4], q, k, v, o, lse, cu), (None, q, k, v, o, lse, cu),
                 (q, q, k, v, o, lse.t(), cu)):
        with pytest.raises(ValueError):
            m.attn_varlen_bwd(*args)
    for kw in (dict(scale=0.0), dict(out=q), dict(scale=float("inf"))):
        with pytest.raises(m.RopeError):
            m.attn_varlen_fwd(q, k, v, cu, **kw)
    with pytest.raises(m.RopeError):                       # 4 query heads do not share 3 key heads
        m.attn_varlen_fwd(q, x[:, :3].contiguous(), x[:, :3].contiguous(), cu)
    with pytest.raises(m.RopeError):
        m.attn_varlen_fwd(*(normal((8, 2, 256), 2, dev) for _ in range(3)), cu)
    with pytest.raises(m.RopeError):
        m.attn_varlen_bwd(o, q, k, v, o, lse, cu, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    cache, table, _, _ = make_paged(dev, [8], 16, 2, 64, 3)
    lens = torch.tensor([8], dtype=torch.int32, device=dev)
    for args in ((q.float(), cache, table, lens, cu), (q, None, table, lens, cu), (q, cache, table.long(), lens, cu),
                 (q, cache, table, lens.long(), cu), (q, cache, table, lens, cu.cpu()),
                 (normal((8, 4, 128), 4, dev), cache, table, lens, cu)):
        with pytest.raises(ValueError):
            m.attn_paged(*args)


def test_results_do_not_depend_on_what_no_row_sees(dev):
    """The same bits whatever lies in other samples, past seq_used and in stale cache slots."""
    m = pr()
    used = [77, 150, 1]
    cu = torch.tensor([3, 103, 303, 310], dtype=torch.int32, device=dev)
    su = torch.tensor(used, dtype=torch.int32, device=dev)
    inside = torch.zeros(320, dtype=torch.bool, device=dev)
    for a, n in zip([3, 103, 303], used):
        inside[a:a + n] = True
    base = [normal((320, h, 64), 5 + i, dev) for i, h in enumerate((6, 2, 2, 6))]
    first = None
    for fill in (0.0, 1e30, float("nan"), float("-inf")):
        q, k, v, dout = (x.clone() for x in base)
        for x in (q, k, v, dout):
            x[~inside] = fill
        o, lse = m.attn_varlen_fwd(q, k, v, cu, seq_used=su, return_lse=True)
        now = (o, lse, *m.attn_varlen_bwd(dout, q, k, v, o, lse, cu, seq_used=su))
        torch.cuda.synchronize()
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now
    for new in (1, 40):
        first = None
        qn = normal((new, 6, 64), 9, dev)
        for fill in (0.0, 1e30, float("nan"), float("inf")):
            cache, table, _, _ = make_paged(dev, [203], 24, 2, 64, 6, fill=fill)
            now = m.attn_paged(qn, cache, table, torch.tensor([203], dtype=torch.int32, device=dev),
                               torch.tensor([0, new], dtype=torch.int32, device=dev))
            assert first is None or torch.equal(first, now)
            first = now


def test_few_key_tiles_shared_by_a_cluster(dev):
    """Backward of problems with few tiles of keys and many streamed ones."""
    check_varlen(dev, [600], 16, 1, 64, True, seed=110)
    check_varlen(dev, [1100], 8, 1, 128, False, seed=111)
    check_varlen(dev, [400, 300], 12, 2, 128, True, seed=112, lead=3, tail=1)
    check_varlen(dev, [500, 0, 260], 40, 1, 80, True, seed=113, used=[499, 0, 200])


def test_key_tiles_shared_over_two_rounds(dev):
    """More CTAs than SMs: causal samples of many tiles in pairs and by four, uneven and long."""
    check_varlen(dev, [1500], 32, 8, 128, True, seed=114)
    check_varlen(dev, [4000], 8, 2, 64, True, seed=115)
    check_varlen(dev, [1, 3900, 2, 3301], 8, 1, 80, True, seed=116, used=[1, 3000, 0, 3301], lead=1, tail=2)


def test_example_runs(dev):
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, os.path.join(root, "examples", "attention_layer.py")], capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert "served in" in out.stdout
