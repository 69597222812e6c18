"""Offsets and lengths that are invalid (needs a GB300): every buffer that a call writes lies between
guards, and they stay as they were."""
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


class Guarded:
    """Buffers with 64 KB of a pattern on either side."""

    PAD = 1 << 16

    def __init__(self, dev):
        self.dev, self.made = dev, []

    def __call__(self, shape, dtype):
        n = dtype.itemsize * torch.Size(shape).numel()
        whole = torch.full((2 * self.PAD + n,), 0x5a, dtype=torch.uint8, device=self.dev)
        self.made.append(whole)
        return whole[self.PAD:self.PAD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for x in self.made:
            assert bool((x[:self.PAD] == 0x5a).all()) and bool((x[-self.PAD:] == 0x5a).all())


OFFSETS = ([0, 150, 90, 200], [-40, 60, 120], [0, 90, 5000], [300, 400, 500], [200, 100, 0], [0, 0, 2 ** 31 - 1],
           [-2 ** 31, 200])


@pytest.mark.parametrize("cu_list", OFFSETS, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_packed(dev, cu_list, causal):
    from packed_varlen_rope_gb300 import _attention as A
    from packed_varlen_rope_gb300 import attn_fault, attn_varlen_bwd, load_library

    A._load_torch()
    T, hq, hkv, d = 200, 4, 2, 64
    q, k, v = qkv_views(T, hq, hkv, d, 300, dev, "fused")
    dout = normal((T, hq, d), 301, dev)
    cu = torch.tensor(cu_list, dtype=torch.int32, device=dev)
    for used in (None, [10 ** 9, -5, 150][:len(cu_list) - 1]):
        su = None if used is None else torch.tensor(used, dtype=torch.int32, device=dev)
        new = Guarded(dev)
        out, lse = new((T, hq, d), torch.bfloat16), new((hq, T), torch.float32)
        dq, dk, dv = new((T, hq, d), torch.bfloat16), new((T, hkv, d), torch.bfloat16), new((T, hkv, d), torch.bfloat16)
        ws = new((T * hq * 8,), torch.uint8)
        desc, at = A._varlen_desc(q, k, v, out, lse, cu, causal, None, su)
        A._launch(load_library().attn_varlen_fwd, "attn_varlen_fwd", at, None, desc)
        attn_varlen_bwd(dout, q, k, v, out, lse, cu, causal=causal, seq_used=su, dq=dq, dk=dk, dv=dv, workspace=ws)
        new.check()
        assert not attn_fault()


@pytest.mark.parametrize("cu_list", OFFSETS, ids=str)
@pytest.mark.parametrize("T,page", [(200, 24), (4, 64)])
def test_paged(dev, cu_list, T, page):
    from packed_varlen_rope_gb300 import PagedKVCache, attn_fault, attn_paged, attn_paged_workspace_bytes, rope_kv_append

    hq, hkv, d, n = 4, 2, 64, len(cu_list) - 1
    if T == 4:
        cu_list = [max(-2 ** 31, x // 50) for x in cu_list]
    cache, table, _, _ = make_paged(dev, [4000] * n, page, hkv, d, 302)
    cu = torch.tensor(cu_list, dtype=torch.int32, device=dev)
    q = normal((T, hq, d), 303, dev)
    k, v = normal((T, hkv, d), 304, dev), normal((T, hkv, d), 305, dev)
    for lens in ([2 ** 31 - 1, -2 ** 31, 4000], [4000, 100, 3]):
        lens = torch.tensor(lens[:n], dtype=torch.int32, device=dev)
        new = Guarded(dev)
        out, q_out = new((T, hq, d), torch.bfloat16), new((T, hq, d), torch.bfloat16)
        shape = tuple(cache.k_pages.shape)
        own = PagedKVCache(new(shape, torch.bfloat16), new(shape, torch.bfloat16))
        rope_kv_append(q, k, v, own, table, lens, cu, 1e4, q_out=q_out)
        need = attn_paged_workspace_bytes(q, own, table, lens, cu)
        ws = new((max(need, 16),), torch.uint8)
        attn_paged(q, own, table, lens, cu, out=out, workspace=ws[:need] if need else None)
        new.check()
        assert not attn_fault()
