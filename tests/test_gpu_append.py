"""rope_kv_append against the rotation's own definition, bit for bit (needs a GB300): the
rotated rows must carry exactly the oracle's bits, and nothing else in the cache changes."""
from __future__ import annotations

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import assert_within, causal_mask, normal, offsets, sample_reference  # noqa: E402
from parity_util import to_bits  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from packed_varlen_rope_gb300 import build

    build.build()
    oracle.build()
    return torch.device("cuda:0")


def pr():
    import packed_varlen_rope_gb300 as m

    return m


def pools(n_pages, page, hkv, d, dev, layout, seed=77):
    if layout == "one-pool":
        pool = normal((n_pages, 2, page, hkv, d), seed, dev)
        return pool[:, 0], pool[:, 1]
    if layout == "heads-first":
        return tuple(normal((n_pages, hkv, page, d), seed + i, dev).transpose(1, 2) for i in range(2))
    return tuple(normal((n_pages, page, hkv, d), seed + i, dev) for i in range(2))


def run_case(dev, new, kv, page, hq, hkv, d, theta=1e6, layout="plain", in_place=False, cached=0, scale=1.0, lead=0,
             tail=0, table_edit=None, seed=1, head_major=False):
    m = pr()
    cu_list = offsets(new, lead)
    T = cu_list[-1] + tail
    x = normal((T, hq + 2 * hkv, d), seed, dev)
    if head_major:
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    need = [-(-max(n, 0) // page) for n in kv]
    n_pages = sum(need) + 4
    kp, vp = pools(n_pages, page, hkv, d, dev, layout)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(kv), max(need + [1])), 1 << 30, dtype=torch.int32)
    for s, n in enumerate(need):
        for i in range(n):
            table[s, i] = order.pop()
    if table_edit:
        table_edit(table, n_pages)
    q0, k0, v0 = (to_bits(t.contiguous()) for t in (q, k, v))
    want_k, want_v = to_bits(kp.contiguous()).copy(), to_bits(vp.contiguous()).copy()
    want_q = q0.copy()
    orc = oracle.get()
    for s, (a, n) in enumerate(zip(cu_list, new)):
        if n == 0:
            continue
        pos = np.arange(n) + kv[s] - n
        pos = np.where((pos >= 0) & (pos < 1 << 24), pos, -1).astype(np.int32)
        want_q[a:a + n] = orc.rope_rows(q0[a:a + n], pos, theta, scale=scale)
        kr = orc.rope_rows(k0[a:a + n], pos, theta, scale=scale)
        for i in range(n):
            if pos[i] < 0 or pos[i] // page >= table.shape[1]:
                continue
            at = int(table[s, pos[i] // page])
            if 0 <= at < n_pages:
                want_k[at, pos[i] % page], want_v[at, pos[i] % page] = kr[i], v0[a + i]
    cs = m.new_cos_sin_cache(cached, d, theta, device=dev, position_scale=scale) if cached else None
    out = None if in_place else torch.zeros((T, hq, d), dtype=torch.bfloat16, device=dev)
    got = m.rope_kv_append(q, k, v, m.PagedKVCache(kp, vp), table.to(dev),
                           torch.tensor(kv, dtype=torch.int32, device=dev),
                           torch.tensor(cu_list, dtype=torch.int32, device=dev), theta, q_out=out, position_scale=scale,
                           cos_sin_cache=cs)
    torch.cuda.synchronize()
    assert np.array_equal(to_bits(got.contiguous()), want_q)
    assert np.array_equal(to_bits(kp.contiguous()), want_k) and np.array_equal(to_bits(vp.contiguous()), want_v)
    assert np.array_equal(to_bits(k.contiguous()), k0) and np.array_equal(to_bits(v.contiguous()), v0)
    if not in_place:
        assert np.array_equal(to_bits(q.contiguous()), q0)


@pytest.mark.parametrize("layout", ["plain", "heads-first", "one-pool"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [8, 24, 64])
def test_layouts(dev, layout, in_place, page):
    run_case(dev, [1, 30, 0, 5], [40, 30, 9, 1000], page, 8, 2, 128, layout=layout, in_place=in_place, lead=2, tail=3)


@pytest.mark.parametrize("d", [16, 48, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (40, 8)])
def test_heads(dev, d, hq, hkv):
    run_case(dev, [3, 1, 70], [3, 513, 200], 16, hq, hkv, d, theta=1e4, seed=3)


@pytest.mark.parametrize("cached", [0, 1, 600, 2000])
def test_cos_sin_cache_and_scale(dev, cached):
    run_case(dev, [1, 20], [1500, 610], 32, 4, 2, 64, cached=cached, seed=4)
    run_case(dev, [1, 20], [1500, 610], 32, 4, 2, 64, cached=cached, scale=4.0, seed=5, in_place=True, head_major=True)


def test_positions_left_out(dev):
    """Negative positions, positions past 2^24, pages past the table or outside the pool."""
    run_case(dev, [5, 2], [3, 2], 8, 4, 2, 64, seed=6)
    run_case(dev, [4, 2], [-10, 2], 8, 4, 2, 64, seed=6, in_place=True)

    def spoil(table, n_pages):
        table[0, 1], table[1, 0] = -1, n_pages

    run_case(dev, [30, 9], [40, 9], 8, 4, 2, 64, seed=7, table_edit=spoil)


def test_many_sequences(dev):
    run_case(dev, [1] * 700, [1 + (91 * i) % 300 for i in range(700)], 16, 4, 1, 64, seed=8)
    run_case(dev, [1] * 255, [1 + (91 * i) % 300 for i in range(255)], 16, 4, 1, 64, seed=9)


def test_refusals(dev):
    m = pr()
    x = normal((4, 8, 64), 1, dev)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    cache = m.new_paged_kv_cache(6, 16, 2, 64, device=dev)
    table = torch.zeros((1, 2), dtype=torch.int32, device=dev)
    lens = torch.tensor([4], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 4], dtype=torch.int32, device=dev)
    for bad in (dict(cache=m.new_paged_kv_cache(6, 16, 1, 64, device=dev)),
                dict(cache=m.new_paged_kv_cache(6, 16, 2, 128, device=dev)), dict(cache=None),
                dict(page_table=table.long()), dict(page_table=table[0]), dict(kv_lens=lens.long()),
                dict(kv_lens=torch.zeros(2, dtype=torch.int32, device=dev)), dict(cu_seqlens=cu.cpu()),
                dict(q=q.float()), dict(v=x[:, 5:]), dict(q_out=q[:2]),
                dict(cos_sin_cache=torch.zeros((4, 4, 4, 4), device=dev))):
        args = dict(q=q, k=k, v=v, cache=cache, page_table=table, kv_lens=lens, cu_seqlens=cu, theta=1e4)
        with pytest.raises((ValueError, m.RopeError)):
            m.rope_kv_append(**{**args, **bad})
    with pytest.raises(m.RopeError):                       # theta of another cache
        m.rope_kv_append(q, k, v, cache, table, lens, cu, 1e4, cos_sin_cache=m.new_cos_sin_cache(8, 64, 1e6, device=dev))
    with pytest.raises(m.RopeError):                       # q_out over k
        m.rope_kv_append(x[:, 4:6], k, v, cache, table, lens, cu, 1e4)
    with pytest.raises(m.RopeError):                       # values over keys
        m.rope_kv_append(q, k, v, m.PagedKVCache(cache.k_pages, cache.k_pages), table, lens, cu, 1e4)
    with pytest.raises(m.RopeError):                       # a page size that is no multiple of 8
        m.rope_kv_append(q, k, v, m.new_paged_kv_cache(6, 12, 2, 64, device=dev), table, lens, cu, 1e4)


def test_serving_loop(dev):
    """Prompts in chunks, then single tokens: append and attend step by step give what the
    packed attention gives on the whole rotated prompts."""
    m = pr()
    lengths, hq, hkv, d, page, theta = [75, 200, 9], 8, 2, 64, 16, 1e4
    total = sum(lengths)
    cu_all = offsets(lengths)
    x = normal((total, hq + 2 * hkv, d), 30, dev)
    cache = m.new_paged_kv_cache(sum(-(-n // page) for n in lengths), page, hkv, d, device=dev)
    cache.k_pages.fill_(float("nan"))
    cache.v_pages.fill_(float("nan"))
    width = max(-(-n // page) for n in lengths)
    table = torch.zeros((3, width), dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(lengths):
        need = -(-n // page)
        table[s, :need] = torch.arange(at, at + need, dtype=torch.int32, device=dev)
        at += need
    out = torch.empty((total, hq, d), dtype=torch.bfloat16, device=dev)
    done = [0, 0, 0]
    step = 0
    while any(a < b for a, b in zip(done, lengths)):
        new = [min(b - a, (60, 1, 7)[(step + s) % 3]) for s, (a, b) in enumerate(zip(done, lengths))]
        rows = torch.cat([torch.arange(cu_all[s] + done[s], cu_all[s] + done[s] + n, device=dev)
                          for s, n in enumerate(new)])
        y = x[rows].contiguous()
        done = [a + n for a, n in zip(done, new)]
        cu = torch.tensor(offsets(new), dtype=torch.int32, device=dev)
        lens = torch.tensor(done, dtype=torch.int32, device=dev)
        q = m.rope_kv_append(y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], cache, table, lens, cu, theta)
        out[rows] = m.attn_paged(q, cache, table, lens, cu)
        step += 1
    cu = torch.tensor(cu_all, dtype=torch.int32, device=dev)
    whole = x.clone()
    m.rope_qk_fwd(*(q := (whole[:, :hq].contiguous(), whole[:, hq:hq + hkv].contiguous())), cu, theta)
    for s, n in enumerate(lengths):
        a = cu_all[s]
        ref = sample_reference(q[0][a:a + n], q[1][a:a + n], whole[a:a + n, hq + hkv:], d ** -0.5,
                               causal_mask(n, n, True, dev))
        assert_within(out[a:a + n], *ref["o"], "o of prompt %d" % s)
