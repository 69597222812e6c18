"""A serving step's page tables against a plain Python walk (needs a GB300): every array, whole."""
from __future__ import annotations

import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from axes_util import NEGATIVE, NO_PAGES, STACK_FULL, TABLE_FULL, TOKENS_PAST_END, step  # noqa: E402


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


def batch(n, page, width, ctx, fresh, over, spare, seed, holes=0.0):
    """(free, count, table, past, new, finished): pages of a pool handed out at random."""
    rng = random.Random(seed)
    past = [rng.randint(0, ctx) for _ in range(n)]
    new = [rng.randint(0, fresh) for _ in range(n)]
    done = [int(rng.random() < over) for _ in range(n)]
    held = [min(-(-p // page), width) for p in past]
    ids = list(range(sum(held) + spare))
    rng.shuffle(ids)
    table = [[rng.choice([-5, -1, 7]) for _ in range(width)] for _ in range(n)]
    for i, h in enumerate(held):
        for j in range(h):
            table[i][j] = -1 if rng.random() < holes else ids.pop()
    count = len(ids)
    return ids + [0] * sum(held), count, table, past, new, done


def check(dev, free, count, table, past, new, finished, page, max_tokens, stride=0, alias=False, stream=None):
    m = pr()
    want = step(free, count, table, past, new, page, max_tokens, finished)
    n, width = len(past), len(table[0]) if table else 3
    pool = torch.full((n, width + stride), 99, dtype=torch.int32, device=dev)
    t = pool[:, :width]
    if n:
        t.copy_(ints(table, dev))
    f, c = ints(free, dev), ints([count], dev)
    out = c if alias else ints([-3], dev)
    status = ints([-1], dev)
    cu, kv, slots = m.paged_kv_step(f, c, t, ints(past, dev), ints(new, dev), page, max_tokens,
                                    finished=None if finished is None else ints(finished, dev),
                                    count_out=None if alias else out, status=status, stream=stream)
    torch.cuda.synchronize()
    assert f.tolist() == want["free"]
    assert out.tolist() == [want["count"]]
    assert (t.tolist() if n else []) == want["table"]
    assert cu.tolist() == want["cu"] and kv.tolist() == want["kv"]
    assert (slots.tolist() if max_tokens else []) == want["slots"]
    assert status.tolist() == [want["status"]], (status.tolist(), want["status"])
    assert bool((pool[:, width:] == 99).all())
    return want


@pytest.mark.parametrize("n", [0, 1, 2, 31, 33, 64, 511, 512, 513, 1025, 3000, 4097, 9000])
@pytest.mark.parametrize("fresh", [1, 40])
def test_steps(dev, n, fresh):
    free, count, table, past, new, done = batch(n, 16, 30, 300, fresh, 0.2, 4 * n + 9, n + fresh)
    total = sum(new)
    check(dev, free, count, table, past, new, done, 16, total + 7, alias=n % 2 == 0)
    check(dev, free, count, table, past, new, None, 16, total, stride=5)


@pytest.mark.parametrize("page", [1, 7, 8, 24, 64, 65536])
def test_page_sizes(dev, page):
    free, count, table, past, new, done = batch(77, page, max(3, 500 // page), 300, 150, 0.3, 77 * (150 // page + 2), page)
    check(dev, free, count, table, past, new, done, page, 77 * 150)


@pytest.mark.parametrize("max_tokens", [0, 1, 512, 513, 2048, 2049, 16384, 16385, 70000])
def test_tokens_of_one_and_two_launches(dev, max_tokens):
    free, count, table, past, new, done = batch(3, 32, 900, 9000, 9000, 0.0, 1000, 5)
    check(dev, free, count, table, past, new, done, 32, max_tokens)
    check(dev, free, count, table, past, [0, 0, 0], done, 32, max_tokens)
    free, count, table, past, new, done = batch(1, 32, 900, 9000, 9000, 0.0, 1000, 13)
    check(dev, free, count, table, past, new, done, 32, max_tokens)
    free, count, table, past, new, done = batch(1500, 8, 9, 30, 1, 0.2, 30000, 14)
    check(dev, free, count, table, past, new, done, 8, max_tokens)
    free, count, table, past, new, done = batch(7000, 8, 9, 30, 12, 0.2, 30000, 6)
    check(dev, free, count, table, past, new, done, 8, max_tokens)


def test_what_does_not_fit_is_reported(dev):
    base = batch(200, 8, 12, 80, 10, 0.0, 30, 7)
    want = check(dev, *base[:5], base[5], 8, 2000)
    assert want["status"] & NO_PAGES and want["status"] & TABLE_FULL == 0
    want = check(dev, *batch(200, 8, 8, 80, 10, 0.2, 500, 8)[:5], None, 8, 2000)
    assert want["status"] & TABLE_FULL
    free, count, table, past, new, done = batch(200, 8, 12, 80, 10, 0.5, 500, 9)
    want = check(dev, free[:count + 20], count, table, past, new, done, 8, 300)
    assert want["status"] & STACK_FULL and want["status"] & TOKENS_PAST_END
    past[3], new[5], past[9] = -4, -1, -(1 << 31)
    assert check(dev, free, count, table, past, new, done, 8, 2000)["status"] & NEGATIVE
    assert check(dev, free, 0, table, past, new, None, 8, 2000)["status"] & NO_PAGES


def test_holes_do_not_go_back(dev):
    free, count, table, past, new, done = batch(700, 8, 70, 500, 10, 0.4, 2000, 10, holes=0.3)
    check(dev, free, count, table, past, new, done, 8, 4000)


def test_lengths_out_of_range_stay_inside(dev):
    """Lengths that no cache has: the arrays are not left, and the step ends."""
    m = pr()
    for n in (3, 2000):
        big = ints([(1 << 31) - 1] * n, dev)
        table, status = torch.zeros((n, 4), dtype=torch.int32, device=dev), ints([0], dev)
        free = torch.arange(100, dtype=torch.int32, device=dev)
        for tokens in (50, 40000):
            cu, kv, slots = m.paged_kv_step(free, ints([100], dev), table, big, big, 8, tokens, status=status,
                                            finished=ints([i % 2 for i in range(n)], dev))
            assert kv.tolist() == [(1 << 31) - 1] * n and cu.tolist()[-1] == (1 << 31) - 1
            assert status.item() & (TABLE_FULL | TOKENS_PAST_END) == TABLE_FULL | TOKENS_PAST_END


@pytest.mark.parametrize("tokens", [60, 500, 700, 3000])
def test_slots_beside_a_length_that_no_cache_has(dev, tokens):
    """A row whose length, and a sum of lengths, that stop at 2^31 - 1: what the table holds of it, and the
    rows before it, have their slots all the same."""
    m, page, width, end = pr(), 8, 40, (1 << 31) - 1
    for past, new in (([0, 20], [10, end]), ([5, end], [3, 100]), ([0, 320, 0], [30, 10, end]), ([0, end, 0], [30, end, 50])):
        n = len(past)
        table = [[100 * i + j if j < -(-p // page) else -1 for j in range(width)] for i, p in enumerate(past)]
        t, free = ints(table, dev), list(range(1000, 1100))
        cu, kv, slots = m.paged_kv_step(ints(free, dev), ints([100], dev), t, ints(past, dev), ints(new, dev), page, tokens)
        want, top = [], list(free)
        for i in range(n):
            for j in range(min(-(-past[i] // page), width), min(-(-(past[i] + new[i]) // page), width)):
                table[i][j] = top.pop()
            for q in range(past[i], past[i] + min(new[i], tokens)):
                want.append(table[i][q // page] * page + q % page if q // page < width else -1)
        assert t.tolist() == table and slots.tolist() == (want + [-1] * tokens)[:tokens]
        assert kv.tolist() == [min(p + x, end) for p, x in zip(past, new)]


def test_a_run_of_steps_in_a_graph(dev):
    """Captured once with the count updated in place, replayed for several steps of a batch
    whose sequences grow, end and are replaced."""
    m, rng = pr(), random.Random(11)
    n, page, width = 50, 8, 20
    free, count, table = list(range(400)), 400, [[-1] * width for _ in range(n)]
    f, c, t = ints(free, dev), ints([count], dev), ints(table, dev)
    past, new, done = (torch.zeros(n, dtype=torch.int32, device=dev) for _ in range(3))
    cu, kv = torch.zeros(n + 1, dtype=torch.int32, device=dev), torch.zeros(n, dtype=torch.int32, device=dev)
    slots, status = torch.zeros(900, dtype=torch.int64, device=dev), ints([0], dev)
    call = lambda: m.paged_kv_step(f, c, t, past, new, page, finished=done, cu_seqlens=cu, kv_lens=kv, slots=slots,   # noqa: E731
                                   status=status)
    call()                                                   # nothing grows: nothing changes
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    lens = [0] * n
    for _ in range(12):
        grow = [rng.randint(0, 17) for _ in range(n)]
        over = [int(x + g > width * page - 20 or rng.random() < 0.1) for x, g in zip(lens, grow)]
        past.copy_(ints(lens, dev)), new.copy_(ints(grow, dev)), done.copy_(ints(over, dev))
        graph.replay()
        want = step(free, count, table, lens, grow, page, 900, over)
        free, count, table, lens = want["free"], want["count"], want["table"], want["kv"]
        assert c.tolist() == [count] and f.tolist() == free and t.tolist() == table
        assert cu.tolist() == want["cu"] and kv.tolist() == lens and slots.tolist() == want["slots"]
        assert status.item() == want["status"]


def test_another_stream(dev):
    side = torch.cuda.Stream(dev)
    free, count, table, past, new, done = batch(100, 16, 30, 300, 3, 0.2, 500, 12)
    torch.cuda.synchronize()
    check(dev, free, count, table, past, new, done, 16, 400, stream=side)


def test_refusals(dev):
    m = pr()
    base = dict(free_pages=ints([1, 2, 3], dev), free_count=ints([3], dev), page_table=ints([[0, 0]], dev),
                past_lens=ints([0], dev), new_lens=ints([1], dev), page_size=8, max_tokens=4)
    m.paged_kv_step(**base)
    for bad in (dict(page_table=base["page_table"].long()), dict(page_table=ints([0, 0], dev)),
                dict(page_table=base["page_table"].cpu()), dict(past_lens=ints([0, 0], dev)),
                dict(new_lens=ints([1], dev, torch.int64)), dict(free_count=ints([1, 2], dev)),
                dict(finished=torch.zeros(1, dtype=torch.bool, device=dev)), dict(slots=ints([0], dev)),
                dict(kv_lens=ints([0, 0], dev)), dict(cu_seqlens=ints([0], dev)), dict(status=ints([0, 0], dev))):
        with pytest.raises(ValueError):
            m.paged_kv_step(**{**base, **bad})
    for bad in (dict(page_size=0), dict(page_size=1 << 17), dict(kv_lens=base["past_lens"]),
                dict(count_out=base["new_lens"]), dict(status=base["free_count"])):
        with pytest.raises(m.RopeError):
            m.paged_kv_step(**{**base, **bad})
