"""The rotation by several position axes against its definition, bit for bit (needs a GB300)."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import normal, offsets  # noqa: E402
from axes_util import rotate  # noqa: E402
from parity_util import to_bits  # noqa: E402


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


def positions(n_axes, T, seed, top=5000):
    rng = np.random.default_rng(seed)
    return rng.integers(0, top, size=(n_axes, T))


def inputs(T, hq, hkv, d, seed, dev, head_major=False):
    x = normal((T, hq + 2 * hkv, d), seed, dev)
    if head_major:
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def run_case(dev, T, hq, hkv, sections, theta=1e6, interleaved=False, own=False, wide=False, backward=False,
             in_place=False, cached=0, scale=1.0, seed=1, head_major=False, pos=None):
    m, d = pr(), 2 * sum(sections)
    q, k, _ = inputs(T, hq, hkv, d, seed, dev, head_major)
    pos = positions(len(sections), T, seed) if pos is None else pos
    ids = torch.from_numpy(pos.astype(np.int64 if wide else np.int32)).to(dev)
    q0, k0 = to_bits(q.contiguous()), to_bits(k.contiguous())
    rule = dict(interleaved=interleaved, own=own, scale=scale, bwd=backward)
    want_q, want_k = (rotate(x, pos, theta, sections, **rule) for x in (q0, k0))
    cs = m.new_cos_sin_cache(cached, d, theta, device=dev, position_scale=scale) if cached else None
    out = {} if in_place else dict(q_out=torch.zeros((T, hq, d), dtype=torch.bfloat16, device=dev),
                                   k_out=torch.zeros((T, hkv, d), dtype=torch.bfloat16, device=dev))
    gq, gk = m.rope_axes_apply(q, k, theta, sections, ids, backward=backward, position_scale=scale, cos_sin_cache=cs,
                               interleaved=interleaved, own_frequencies=own, **out)
    torch.cuda.synchronize()
    assert np.array_equal(to_bits(gq.contiguous()), want_q) and np.array_equal(to_bits(gk.contiguous()), want_k)
    if not in_place:
        assert np.array_equal(to_bits(q.contiguous()), q0) and np.array_equal(to_bits(k.contiguous()), k0)


@pytest.mark.parametrize("T", [1, 2, 17, 1000])
@pytest.mark.parametrize("sections", [(16, 24, 24), (20, 20), (3, 9, 2, 18), (64,), (1, 7), (100, 20, 8)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (7, 1), (32, 8)])
def test_sections(dev, T, sections, hq, hkv):
    run_case(dev, T, hq, hkv, sections, seed=T)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("backward,in_place", [(False, True), (True, False), (True, True)])
def test_forms(dev, interleaved, own, wide, backward, in_place):
    run_case(dev, 333, 6, 2, (24, 20, 20), interleaved=interleaved, own=own, wide=wide, backward=backward,
             in_place=in_place, seed=2, head_major=in_place)
    run_case(dev, 61, 5, 5, (11, 13), theta=1e4, interleaved=interleaved, own=own, wide=wide, backward=backward,
             in_place=in_place, seed=3)


@pytest.mark.parametrize("cached", [0, 1, 600, 6000])
def test_cos_sin_cache_and_scale(dev, cached):
    run_case(dev, 200, 4, 2, (16, 24, 24), cached=cached, seed=4, interleaved=True)
    run_case(dev, 200, 4, 2, (16, 24, 24), cached=cached, seed=5, scale=4.0, backward=True)


def test_far_and_left_out_positions(dev):
    pos = positions(3, 64, 6, 1 << 24)
    pos[0, 3], pos[1, 4], pos[2, 5], pos[2, 6], pos[0, 7] = -1, -7, 1 << 24, (1 << 24) - 1, 0
    for in_place in (False, True):
        run_case(dev, 64, 4, 2, (16, 24, 24), pos=pos, in_place=in_place, seed=7)
        run_case(dev, 64, 4, 2, (16, 24, 24), pos=pos + (pos == 1 << 24) * (1 << 40), wide=True, in_place=in_place, seed=7)


def test_equal_positions_give_the_bits_of_one_axis(dev):
    m = pr()
    q, k, _ = inputs(999, 8, 2, 128, 8, dev)
    ids = torch.randint(0, 1 << 20, (999,), device=dev, dtype=torch.int32)
    want = m.rope_qk_apply(q, k, 1e6, position_ids=ids, q_out=torch.empty((999, 8, 128), dtype=q.dtype, device=dev),
                           k_out=torch.empty((999, 2, 128), dtype=q.dtype, device=dev))
    for interleaved in (False, True):
        got = m.rope_axes_apply(q.clone(), k.clone(), 1e6, (16, 24, 24), ids.expand(3, 999).contiguous(),
                                interleaved=interleaved)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        got = m.rope_axes_apply(q.clone(), k.clone(), 1e6, (16, 24, 24), ids[None].expand(3, 999), interleaved=interleaved)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def append_case(dev, new, kv, page, hq, hkv, sections, seed, in_place=False, cached=0, wide=False, table_edit=None,
                pos_edit=None, **rule):
    m, d, theta = pr(), 2 * sum(sections), 1e6
    cu = offsets(new, 2)
    T = cu[-1] + 3
    q, k, v = inputs(T, hq, hkv, d, seed, dev)
    need = [-(-max(n, 0) // page) for n in kv]
    n_pages = sum(need) + 4
    kp, vp = (normal((n_pages, page, hkv, d), seed + i, dev) for i in (50, 51))
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(kv), max(need + [1])), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        for i in range(n):
            table[s, i] = order.pop()
    if table_edit:
        table_edit(table, n_pages)
    pos = positions(len(sections), T, seed)
    if pos_edit:
        pos_edit(pos)
    q0, k0, v0 = (to_bits(t.contiguous()) for t in (q, k, v))
    want_k, want_v = to_bits(kp).copy(), to_bits(vp).copy()
    where = np.full(T, -1)
    for s, (a, n) in enumerate(zip(cu, new)):
        where[a:a + n] = np.arange(n) + kv[s] - n
    ids = np.where((where >= 0) & (where < 1 << 24), pos, -1)       # rows of no place are left out
    want_q, kr = (rotate(x, ids, theta, sections, rule.get("interleaved", False), rule.get("own_frequencies", False))
                  for x in (q0, k0))
    row_ok = ((ids >= 0) & (ids < 1 << 24)).all(axis=0)
    for s, (a, n) in enumerate(zip(cu, new)):
        for t in range(a, a + n):
            if row_ok[t] and where[t] // page < table.shape[1]:
                at = int(table[s, where[t] // page])
                if 0 <= at < n_pages:
                    want_k[at, where[t] % page], want_v[at, where[t] % page] = kr[t], v0[t]
    cs = m.new_cos_sin_cache(cached, d, theta, device=dev) if cached else None
    out = None if in_place else torch.zeros((T, hq, d), dtype=torch.bfloat16, device=dev)
    got = m.rope_kv_append(q, k, v, m.PagedKVCache(kp, vp), table.to(dev), torch.tensor(kv, dtype=torch.int32, device=dev),
                           torch.tensor(cu, dtype=torch.int32, device=dev), theta, q_out=out, cos_sin_cache=cs,
                           position_ids=torch.from_numpy(pos.astype(np.int64 if wide else np.int32)).to(dev),
                           sections=sections, **rule)
    torch.cuda.synchronize()
    assert np.array_equal(to_bits(got.contiguous()), want_q)
    assert np.array_equal(to_bits(kp), want_k) and np.array_equal(to_bits(vp), want_v)
    assert np.array_equal(to_bits(k.contiguous()), k0) and np.array_equal(to_bits(v.contiguous()), v0)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [8, 24, 64])
@pytest.mark.parametrize("cached", [0, 1000])
def test_append(dev, in_place, page, cached):
    append_case(dev, [1, 30, 0, 5], [40, 30, 9, 1000], page, 8, 2, (16, 24, 24), 9, in_place, cached, wide=in_place)
    append_case(dev, [3, 1, 70], [3, 513, 200], page, 40, 8, (20, 20), 10, in_place,
                **({} if cached else dict(own_frequencies=True)))
    append_case(dev, [3, 1, 70], [3, 513, 200], page, 2, 2, (100, 20, 8), 10, in_place, cached, interleaved=True)


def test_append_leaves_rows_out(dev):
    def spoil(table, n_pages):
        table[0, 1], table[1, 0] = -1, n_pages

    def unplaced(pos):
        pos[0, 4], pos[2, 6], pos[1, 9] = -1, 1 << 24, -3

    for in_place in (False, True):
        append_case(dev, [5, 2], [3, 2], 8, 4, 2, (16, 16), 11, in_place)
        append_case(dev, [30, 9], [40, 9], 8, 4, 2, (8, 8, 16), 12, in_place, table_edit=spoil, pos_edit=unplaced)
    append_case(dev, [1] * 700, [1 + (91 * i) % 300 for i in range(700)], 16, 4, 1, (16, 8, 8), 13)


def test_gradients(dev):
    """The rotation is linear and orthogonal: its gradient is the transpose rotation of the incoming
    one, also of broadcast gradients, and rows left out pass theirs on."""
    m = pr()
    q, k, _ = inputs(77, 6, 2, 128, 14, dev)
    pos = positions(3, 77, 14)
    pos[1, 5] = -1
    ids = torch.from_numpy(pos).to(dev)
    q, k = q.detach().clone().requires_grad_(), k.detach().clone().requires_grad_()
    gq, gk = normal((77, 6, 128), 15, dev), normal((1, 1, 128), 16, dev)
    oq, ok = m.apply_rope_axes(q.clone(), k.clone(), 1e6, (16, 24, 24), ids, interleaved=True)
    torch.autograd.backward([oq, ok], [gq, gk.expand(77, 2, 128)])
    for x, g in ((q, gq), (k, gk.expand(77, 2, 128))):
        want = rotate(to_bits(g.contiguous()), pos, 1e6, (16, 24, 24), interleaved=True, bwd=True)
        assert np.array_equal(to_bits(x.grad), want)
    rope = m.RotaryEmbedding(128, 1e6, sections=(16, 24, 24), interleaved=True)
    again = rope(q.detach().clone(), k.detach().clone(), position_ids=ids)
    assert torch.equal(again[0], oq) and torch.equal(again[1], ok)
    with pytest.raises(RuntimeError):
        (g,) = torch.autograd.grad(m.apply_rope_axes(q.clone(), k.detach().clone(), 1e6, (16, 24, 24), ids)[0].float().sum(),
                                   q, create_graph=True)
        g.float().square().sum().backward()


def test_streams_and_graph(dev):
    """Captured and replayed on new values; and on a stream that is not torch's current one."""
    m = pr()
    q, k, _ = inputs(300, 8, 2, 64, 17, dev)
    ids = torch.from_numpy(positions(2, 300, 17)).to(dev)
    out = [torch.empty((300, h, 64), dtype=q.dtype, device=dev) for h in (8, 2)]
    call = lambda s=None: m.rope_axes_apply(q, k, 1e4, (16, 16), ids, q_out=out[0], k_out=out[1], stream=s)   # noqa: E731
    graph = torch.cuda.CUDAGraph()
    call()
    with torch.cuda.graph(graph):
        call()
    for seed in (18, 19):
        pos = positions(2, 300, seed)
        ids.copy_(torch.from_numpy(pos))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(to_bits(out[0]), rotate(to_bits(q.contiguous()), pos, 1e4, (16, 16)))
    side = torch.cuda.Stream(dev)
    out[0].zero_()
    side.wait_stream(torch.cuda.current_stream(dev))
    call(side)
    side.synchronize()
    assert np.array_equal(to_bits(out[0]), rotate(to_bits(q.contiguous()), pos, 1e4, (16, 16)))


def test_offsets_past_32_bits(dev):
    """A view that spans more than 2^31 elements: token strides of 2^27."""
    m = pr()
    pool = torch.zeros((40 << 27,), dtype=torch.bfloat16, device=dev)
    x = pool.as_strided((33, 2, 64), (1 << 27, 64, 1))
    x.copy_(normal((33, 2, 64), 20, dev))
    before, pos = to_bits(x.contiguous()), positions(2, 33, 20)
    m.rope_axes_apply(x[:, :1], x[:, 1:], 1e4, (16, 16), torch.from_numpy(pos).to(dev))
    assert np.array_equal(to_bits(x.contiguous()), rotate(before, pos, 1e4, (16, 16)))


def test_refusals(dev):
    m = pr()
    q, k, v = inputs(9, 4, 2, 64, 21, dev)
    ids = torch.zeros((2, 9), dtype=torch.int32, device=dev)
    cs = m.new_cos_sin_cache(10, 64, 1e4, device=dev)
    for bad in (dict(sections=(16, 15)), dict(sections=(32, 0)), dict(sections=(8, 8, 8, 4, 4)), dict(position_ids=ids[:1]),
                dict(position_ids=ids.float()), dict(position_ids=ids.cpu()), dict(position_ids=ids[:, :8]),
                dict(position_ids=torch.zeros((9, 2), dtype=torch.int32, device=dev).t()), dict(q_out=q.clone()),
                dict(q=q.float()), dict(position_ids=None)):
        args = dict(q=q, k=k, theta=1e4, sections=(16, 16), position_ids=ids)
        args.update(bad)
        with pytest.raises((ValueError, m.RopeError)):
            m.rope_axes_apply(**args)
    for bad in (dict(own_frequencies=True, cos_sin_cache=cs), dict(theta=1e5, cos_sin_cache=cs), dict(k=q[:, :2])):
        args = dict(q=q, k=k, theta=1e4, sections=(16, 16), position_ids=ids)
        args.update(bad)
        with pytest.raises(m.RopeError):
            m.rope_axes_apply(**args)
    cache = m.new_paged_kv_cache(3, 16, 2, 64, device=dev)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device=dev), torch.tensor([9], dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 9], dtype=torch.int32, device=dev)
    for bad in (dict(position_ids=ids), dict(sections=(16, 16)), dict(interleaved=True), dict(own_frequencies=True),
                dict(position_ids=ids, sections=(16, 8))):
        with pytest.raises((ValueError, m.RopeError)):
            m.rope_kv_append(q, k, v, cache, table, lens, cu, 1e4, **bad)
    rope = m.RotaryEmbedding(64, 1e4, sections=(16, 16))
    with pytest.raises(ValueError):
        rope(q, k, cu_seqlens=cu)
    with pytest.raises(ValueError):
        m.RotaryEmbedding(64, 1e4, sections=(16, 8))
