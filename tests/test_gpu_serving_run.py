"""The operators of a serving loop together, as they would be used (needs a GB300): page tables on the
device, rotation by several axes on the way into the cache, attention with rules over it; each step
against attention over whole sequences, also captured in one graph.  And a training layer of them."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import U, assert_within, normal, offsets  # noqa: E402
from axes_util import rotate  # noqa: E402
from parity_util import to_bits  # noqa: E402
from rule_util import sample_reference  # noqa: E402

HQ, HKV, D, PAGE, THETA, SECTIONS = 8, 2, 64, 16, 1e5, (8, 12, 12)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from packed_varlen_rope_gb300 import build

    build.build()
    return torch.device("cuda:0")


def ints(x, dev, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=dev)


def from_bits(bits, dev):
    return torch.from_numpy(bits.view(np.int16)).to(dev).view(torch.bfloat16)


class Loop:
    """Rows of a batch that grow, end and are replaced; everything a step needs is on the device."""

    def __init__(self, dev, rows=5, pages=60, width=12, most=128):
        import packed_varlen_rope_gb300 as pr

        self.pr, self.dev, self.rows, self.most = pr, dev, rows, most
        self.free, self.count = torch.arange(pages, dtype=torch.int32, device=dev), ints([pages], dev)
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
        self.past, self.new, self.over = (torch.zeros(rows, dtype=torch.int32, device=dev) for _ in range(3))
        self.status, self.prefix = ints([0], dev), torch.zeros(rows, dtype=torch.int32, device=dev)
        self.cache = pr.new_paged_kv_cache(pages, PAGE, HKV, D, device=dev)
        self.cache.k_pages.fill_(float("nan")), self.cache.v_pages.fill_(float("nan"))
        self.qkv = torch.zeros((most, HQ + 2 * HKV, D), dtype=torch.bfloat16, device=dev)
        self.ids = torch.full((3, most), -1, dtype=torch.int32, device=dev)
        self.slopes = torch.tensor([2.0 ** (-h) for h in range(1, HQ + 1)], device=dev)
        self.q = torch.zeros((most, HQ, D), dtype=torch.bfloat16, device=dev)
        self.out = torch.zeros_like(self.q)

    def step(self):
        pr = self.pr
        cu, kv, slots = pr.paged_kv_step(self.free, self.count, self.table, self.past, self.new, PAGE, self.most,
                                         finished=self.over, status=self.status)
        x = self.qkv
        pr.rope_kv_append(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.cache, self.table, kv, cu, THETA, q_out=self.q,
                          position_ids=self.ids, sections=SECTIONS, interleaved=True)
        pr.attn_paged(self.q, self.cache, self.table, kv, cu, out=self.out, score_cap=6.0, distance_slopes=self.slopes,
                      prefix_lens=self.prefix)
        return cu, kv, slots


@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(dev, graph):
    loop, rng = Loop(dev), np.random.default_rng(3)
    run, arrays = loop.step, None
    loop.step()                                              # (nothing grows)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            arrays = loop.step()
        run = g.replay
    held = [None] * loop.rows                                # rotated keys and values of every row, and its prefix
    for at in range(14):
        past = [0 if h is None else len(h[0]) for h in held]
        over = [int(h is not None and (len(h[0]) > 90 or rng.random() < 0.15)) for h in held]
        new = [int(rng.integers(0, 30)) if at == 0 or rng.random() < 0.3 else int(rng.integers(0, 3)) for _ in held]
        T = sum(new)
        x = normal((loop.most, HQ + 2 * HKV, D), 100 + at, dev)
        pos = rng.integers(0, 4000, size=(3, loop.most))
        for t, v in ((loop.past, past), (loop.new, new), (loop.over, over)):
            t.copy_(ints(v, dev))
        for i in range(loop.rows):
            if held[i] is None or over[i]:
                held[i] = (torch.zeros((0, HKV, D), dtype=torch.bfloat16, device=dev),) * 2 + (int(rng.integers(0, 20)),)
        loop.prefix.copy_(ints([h[2] for h in held], dev))
        loop.qkv.copy_(x), loop.ids.copy_(torch.from_numpy(pos.astype(np.int32)))
        got = run()
        cu, kv, slots = arrays if graph else got
        torch.cuda.synchronize()
        assert loop.status.item() == 0 and cu.tolist() == offsets(new)
        turned = rotate(to_bits(x[:, :HQ + HKV].contiguous()), pos, THETA, SECTIONS, interleaved=True)
        turned = from_bits(turned, dev)
        flat_k, flat_v = (p.reshape(-1, HKV, D) for p in (loop.cache.k_pages, loop.cache.v_pages))
        for i, (a, n) in enumerate(zip(offsets(new), new)):
            k = torch.cat([held[i][0], turned[a:a + n, HQ:]])
            v = torch.cat([held[i][1], x[a:a + n, HQ + HKV:]])
            held[i] = (k, v, held[i][2])
            assert kv.tolist()[i] == len(k)
            assert torch.equal(flat_k[slots[a:a + n]], k[len(k) - n:]) and torch.equal(flat_v[slots[a:a + n]], v[len(v) - n:])
            if n == 0:
                continue
            ref = sample_reference(turned[a:a + n, :HQ], k, v, D ** -0.5, 6.0, loop.slopes, min(held[i][2], len(k)), True)
            assert_within(loop.out[a:a + n], *ref["o"], "step %d, row %d" % (at, i))
        assert bool((slots[T:] == -1).all()) and not bool(loop.out[T:].any())
    used = [p for row, h in zip(loop.table.tolist(), held) for p in row[:-(-len(h[0]) // PAGE)]]
    left = loop.free.tolist()[:loop.count.item()]
    assert sorted(used + left) == list(range(60))            # every page is one row's, or free
    assert not loop.pr.attn_fault()


def test_training_layer(dev):
    """Rotation by axes, attention with all rules and back again, on the slices of one projection's
    output; pad rows are left out of both."""
    import packed_varlen_rope_gb300 as pr

    lengths, used, prefix = [70, 130, 64], [70, 100, 0], [20, 129, 5]
    cu, T = offsets(lengths), sum(lengths)
    x = normal((T, HQ + 2 * HKV, D), 7, dev)
    leaf = x.clone().requires_grad_()
    slopes = torch.tensor([2.0 ** (-h) for h in range(1, HQ + 1)], device=dev)
    rng = np.random.default_rng(8)
    pos = rng.integers(0, 500, size=(3, T))
    for a, n, u in zip(cu, lengths, used):
        pos[:, a + u:a + n] = -1
    ids = torch.from_numpy(pos).to(dev)
    rope = pr.RotaryEmbedding(D, THETA, sections=SECTIONS)
    q, k = rope(leaf[:, :HQ].clone(), leaf[:, HQ:HQ + HKV].clone(), position_ids=ids)
    o = pr.apply_attn(q, k, leaf[:, HQ + HKV:], ints(cu, dev), seq_used=ints(used, dev), score_cap=5.0, distance_slopes=slopes,
                      prefix_lens=ints(prefix, dev))
    do = normal((T, HQ, D), 9, dev)
    o.backward(do)
    turned = from_bits(rotate(to_bits(x[:, :HQ + HKV].contiguous()), pos, THETA, SECTIONS), dev)
    for a, n, u, pre in zip(cu, lengths, used, prefix):
        assert not bool(o[a + u:a + n].any()) and not bool(leaf.grad[a + u:a + n].any())
        if u == 0:
            continue
        rows = slice(a, a + u)
        ref = sample_reference(turned[rows, :HQ], turned[rows, HQ:], x[rows, HQ + HKV:], D ** -0.5, 5.0, slopes, min(pre, u),
                               True, do[rows])
        assert_within(o[rows], *ref["o"], "o")
        assert_within(leaf.grad[rows, HQ + HKV:], *ref["dv"], "dv")
        # the transpose rotation in binary64: each pair keeps its length, one more rounding to bf16
        # (and that of its input, inside the bound of the pair)
        w = np.power(THETA, -np.arange(D // 2) / (D / 2)).astype(np.float32)
        axis = np.repeat(np.arange(3), SECTIONS)
        phi = torch.from_numpy((pos[axis][:, rows].T.astype(np.float32) * w).astype(np.float64)).to(dev)[:, None, :]
        c, s = phi.cos(), phi.sin()
        for name, cols in (("dq", slice(0, HQ)), ("dk", slice(HQ, HQ + HKV))):
            g, tol = ref[name]
            lo, hi = g.split(D // 2, dim=2)
            want = torch.cat([lo * c + hi * s, hi * c - lo * s], dim=2)
            t0, t1 = tol.split(D // 2, dim=2)
            bound = torch.cat([t0 * c.abs() + t1 * s.abs(), t1 * c.abs() + t0 * s.abs()], dim=2)
            assert_within(leaf.grad[rows, cols], want, bound + U * (want.abs() + bound) + 2.0 ** -20 * g.abs(), name)
