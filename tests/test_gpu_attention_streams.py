"""Explicit streams (needs a GB300): what a call allocates itself comes from the stream it runs on,
so that it never shares memory with work still queued elsewhere."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from attn_util import normal  # noqa: E402
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


class Busy:
    """Queues some tens of milliseconds of products on the current stream."""

    def __init__(self, dev):
        self.a = normal((8192, 8192), 1, dev)
        self.out = torch.empty_like(self.a)

    def __call__(self):
        for _ in range(40):
            torch.mm(self.a, self.a, out=self.out)


def calls(dev):
    """(name, call(stream), sizes in bytes of what it allocates) of every entry point that does."""
    m = pr()
    T, hq, hkv, d = 3000, 8, 2, 128
    q, k, v = qkv_views(T, hq, hkv, d, 200, dev, "plain")
    dout = normal((T, hq, d), 204, dev)
    cu = torch.tensor([0, 1000, T], dtype=torch.int32, device=dev)
    o, lse = m.attn_varlen_fwd(q, k, v, cu, return_lse=True)
    cache, table, _, _ = make_paged(dev, [20000], 64, 1, 128, 205)
    qn = normal((300, 1, 128), 206, dev)
    cun = torch.tensor([0, 300], dtype=torch.int32, device=dev)
    lens = torch.tensor([20000], dtype=torch.int32, device=dev)
    need = m.attn_paged_workspace_bytes(qn, cache, table, lens, cun)
    assert need > 1 << 20
    rows = T * d * 2
    return [("forward", lambda s: m.attn_varlen_fwd(q, k, v, cu, return_lse=True, stream=s), [rows * hq, T * hq * 4]),
            ("backward", lambda s: m.attn_varlen_bwd(dout, q, k, v, o, lse, cu, stream=s),
             [rows * hq, rows * hkv, rows * hkv, T * hq * 8]),
            ("paged", lambda s: (m.attn_paged(qn, cache, table, lens, cun, stream=s),), [qn.numel() * 2, need])]


def other_calls(dev):
    """The same of the rotation's helpers and the GLU."""
    m = pr()
    e, g, dh = (normal((2000, 1024), 220 + i, dev) for i in range(3))
    cu = torch.tensor([0, 300000, 600000], dtype=torch.int32, device=dev)
    phi = torch.rand(600000, generator=torch.Generator(device=dev).manual_seed(223), device=dev) * 1e4
    n = e.numel() * 2
    return [("glu", lambda s: (m.glu_fwd("swiglu", e, g, stream=s),), [n]),
            ("glu backward", lambda s: m.glu_bwd("geglu", dh, e, g, stream=s), [n, n]),
            ("positions", lambda s: (m.rope_qk_positions(cu, 600000, stream=s),), [2400000]),
            ("validation", lambda s: (m.rope_validate_cu_seqlens(cu, 600000, stream=s),), [4]),
            ("cos and sin", lambda s: m.rope_cos_sin_eval(phi, stream=s), [2400000, 2400000]),
            ("cache", lambda s: (m.new_cos_sin_cache(8192, 128, 1e6, device=dev, stream=s).data,), [8192 * 128 * 4])]


@pytest.mark.parametrize("which", [calls, other_calls])
@pytest.mark.parametrize("as_int", [False, True])
def test_memory_freed_behind_queued_work_is_left_alone(dev, as_int, which):
    """Tensors of the very sizes that the call needs, dropped while the current stream has yet to
    read them: their values arrive, and the call's results are right."""
    s, busy = torch.cuda.Stream(), Busy(dev)
    for name, call, sizes in which(dev):
        want = call(None)
        torch.cuda.synchronize()
        olds = [torch.full((n // 4,), 7.0 + i, device=dev) for i, n in enumerate(sizes)]
        busy()
        copies = [x.clone() for x in olds]
        del olds
        got = call(s.cuda_stream if as_int else s)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got)), name
        torch.cuda.synchronize()
        assert all(bool((x == 7.0 + i).all()) for i, x in enumerate(copies)), name


@pytest.mark.parametrize("which", [calls, other_calls])
def test_results_dropped_behind_queued_work_are_left_alone(dev, which):
    """Results of a call on another stream, dropped while the current stream has yet to read them,
    keep their values there although that stream then wants the same sizes."""
    s, busy = torch.cuda.Stream(), Busy(dev)
    for name, call, _ in which(dev):
        want = call(None)
        torch.cuda.synchronize()
        got = call(s)
        s.synchronize()
        busy()
        copies = [x.clone() for x in got]
        del got
        with torch.cuda.stream(s):                        # as the next call there would
            again = [torch.full_like(x, 5.0) for x in want]
        s.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, copies)), name
        assert all(bool((x == 5.0).all()) for x in again)


def test_fault_report_waits_for_every_stream(dev):
    """What attn_fault answers holds for kernels still running on a stream that the default
    stream does not wait for."""
    m = pr()
    T, hq, d = 32768, 16, 128
    q, k, v = qkv_views(T, hq, hq, d, 210, dev, "plain")
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    assert m.attn_fault() is False                       # (loads what it reads)
    torch.cuda.synchronize()
    for _ in range(40):                                  # about 100 ms
        m.attn_varlen_fwd(q, k, v, cu, out=out, stream=s)
    assert not s.query()
    assert m.attn_fault() is False
    assert s.query()
