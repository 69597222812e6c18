"""The host side of the rotation by several axes and of the serving step (no GPU): declarations
against exports, structures against the C compiler's layout, refusals before any launch."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INCLUDE = os.path.join(ROOT, "include")

OK, ERR_NULL, ERR_SHAPE, ERR_HEAD_DIM, ERR_ALIGN, ERR_OVERLAP, ERR_UNSUPPORTED, ERR_LAUNCH, ERR_THETA = \
    0, -1, -2, -3, -4, -5, -6, -7, -8
ERR_CACHE = -11
BASE = 1 << 40                 # made up: no call below follows a pointer


@pytest.fixture(scope="module")
def lib():
    from packed_varlen_rope_gb300 import build, load_library

    build.build()
    return load_library()


def test_exports_match_the_header(lib):
    from packed_varlen_rope_gb300 import PAGED_EXPORTS

    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, "paged_step.h")).read(), flags=re.S)
    assert sorted(PAGED_EXPORTS) == sorted(re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M))
    assert all(hasattr(lib, n) for n in PAGED_EXPORTS)


def test_headers_are_plain_c_and_structures_match(tmp_path):
    from packed_varlen_rope_gb300 import PagedKVStepDesc, RopeAxesDesc

    pairs = (("rope_axes", RopeAxesDesc), ("paged_kv_step_desc", PagedKVStepDesc))
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "rope_axes.h"', '#include "paged_step.h"',
             "int main(void) {"]
    for name, st in pairs:
        lines.append('printf("%%zu\\n", sizeof(%s));' % name)
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (name, f[0]) for f in st._fields_]
    lines.append("return 0; }")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", INCLUDE, str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    want = []
    for _, st in pairs:
        want.append(ctypes.sizeof(st))
        want += [getattr(st, f[0]).offset for f in st._fields_]
    assert got == want


def test_packed_descriptors_fill_the_fields_in_order():
    from packed_varlen_rope_gb300 import PagedKVStepDesc, RopeAxesDesc, RopeQKDesc
    from packed_varlen_rope_gb300 import _axes, _step

    for pack, st in ((_axes._AXES_PACK, RopeAxesDesc), (_axes._QK_PACK, RopeQKDesc), (_step._STEP_PACK, PagedKVStepDesc)):
        assert pack.__self__.size == ctypes.sizeof(st)
    x = RopeAxesDesc.from_buffer_copy(_axes._AXES_PACK(1, 2, 3, 4, 5, 6, 7, 8))
    assert (x.position_ids, x.position_stride, x.n_axes, x.flags, *x.sections) == tuple(range(1, 9))
    q = RopeQKDesc.from_buffer_copy(_axes._QK_PACK(*range(1, 13), 13, 14, 15, 16, 17, 18, 19, 20, 1e4, 2.0, 0, 1, 0, 24, 0, 26, 0))
    assert (q.q, q.q_stride_token, q.q_stride_head, q.k, q.k_stride_token, q.k_stride_head, q.q_out, q.q_out_stride_token,
            q.q_out_stride_head, q.k_out, q.k_out_stride_token, q.k_out_stride_head, q.cu_seqlens, q.n_seqs, q.n_q_heads,
            q.n_kv_heads, q.head_dim, q.position_ids, q.total_tokens, q.token_offset, q.theta, q.position_scale,
            bool(q.cos_sin_cache), q.backward, q.flags, q.seq_used, bool(q.segments), q.n_segments, q.reserved) == \
        (*range(1, 21), 1e4, 2.0, False, 1, 0, 24, False, 26, 0)
    d = PagedKVStepDesc.from_buffer_copy(_step._STEP_PACK(*range(1, 19)))
    assert tuple(getattr(d, f[0]) for f in d._fields_) == tuple(range(1, 19))


def axes(**kw):
    from packed_varlen_rope_gb300 import RopeAxesDesc

    a = RopeAxesDesc(BASE + (1 << 35), 1000, 2, 0, (ctypes.c_int32 * 4)(*kw.pop("sections", (16, 16, 0, 0))))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def rotation(**kw):
    from packed_varlen_rope_gb300 import RopeQKDesc

    p = RopeQKDesc()
    p.q, p.q_stride_token, p.q_stride_head = BASE, 256, 64
    p.k, p.k_stride_token, p.k_stride_head = BASE + (1 << 30), 128, 64
    p.n_q_heads, p.n_kv_heads, p.head_dim, p.total_tokens, p.theta, p.position_scale = 4, 2, 64, 1000, 1e4, 1.0
    for k, v in kw.items():
        assert hasattr(p, k)
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,ax,want", [
    (dict(total_tokens=-1), {}, ERR_SHAPE), (dict(n_q_heads=0), {}, ERR_SHAPE), (dict(head_dim=72), {}, ERR_HEAD_DIM),
    (dict(theta=0.0), {}, ERR_THETA), (dict(position_scale=-1.0), {}, ERR_THETA),
    (dict(cu_seqlens=BASE), {}, ERR_UNSUPPORTED), (dict(position_ids=BASE), {}, ERR_UNSUPPORTED),
    (dict(seq_used=BASE), {}, ERR_UNSUPPORTED), (dict(token_offset=1), {}, ERR_UNSUPPORTED),
    (dict(flags=1), {}, ERR_UNSUPPORTED), (dict(n_segments=1), {}, ERR_UNSUPPORTED), (dict(n_seqs=2), {}, ERR_UNSUPPORTED),
    (dict(q=None), {}, ERR_NULL), (dict(q=BASE + 8), {}, ERR_ALIGN), (dict(k=BASE), {}, ERR_OVERLAP),
    (dict(q_out=BASE + (3 << 30), q_out_stride_token=256, q_out_stride_head=64), {}, ERR_NULL),
    (dict(q_stride_token=64), {}, ERR_OVERLAP), (dict(total_tokens=1 << 31, k=BASE + (1 << 45)), dict(position_stride=1 << 31), ERR_UNSUPPORTED),
    ({}, dict(n_axes=0), ERR_SHAPE), ({}, dict(n_axes=5), ERR_SHAPE), ({}, dict(sections=(16, 15, 0, 0)), ERR_SHAPE),
    ({}, dict(sections=(32, 0, 0, 0)), ERR_SHAPE), ({}, dict(sections=(16, 8, 8, 0)), ERR_SHAPE),
    ({}, dict(sections=(48, -16, 0, 0)), ERR_SHAPE), ({}, dict(flags=8), ERR_UNSUPPORTED),
    ({}, dict(position_ids=None), ERR_NULL), ({}, dict(position_ids=BASE + 2), ERR_ALIGN),
    ({}, dict(position_ids=BASE + 4, flags=4), ERR_ALIGN), ({}, dict(position_stride=-1), ERR_SHAPE),
])
def test_axes_refusals(lib, kw, ax, want):
    assert lib.rope_axes_apply(ctypes.byref(rotation(**kw)), ctypes.byref(axes(**ax)), None) == want


def test_axes_nothing_to_do(lib):
    p = rotation(total_tokens=0, q=None, k=None)
    assert lib.rope_axes_apply(ctypes.byref(p), ctypes.byref(axes(position_ids=None)), None) == OK
    assert lib.rope_axes_apply(None, ctypes.byref(axes()), None) == ERR_NULL
    assert lib.rope_axes_apply(ctypes.byref(p), None, None) == ERR_NULL
    assert lib.rope_kv_append_axes(None, None, None) == ERR_NULL


def test_axes_with_a_cache_of_shared_frequencies(lib):
    from packed_varlen_rope_gb300 import RopeCosSinCacheDesc

    cs = RopeCosSinCacheDesc()
    p = rotation()
    p.cos_sin_cache = ctypes.pointer(cs)
    assert lib.rope_axes_apply(ctypes.byref(p), ctypes.byref(axes(flags=2)), None) == ERR_CACHE
    assert lib.rope_axes_apply(ctypes.byref(p), ctypes.byref(axes()), None) == ERR_CACHE      # never built


def test_append_refusals(lib):
    from test_attn_abi_host import append

    good = append()                                          # heads of 64
    for ax, want in ((dict(sections=(16, 8, 0, 0)), ERR_SHAPE), (dict(position_ids=None), ERR_NULL),
                     (dict(n_axes=9), ERR_SHAPE), (dict(flags=64), ERR_UNSUPPORTED)):
        assert lib.rope_kv_append_axes(ctypes.byref(good), ctypes.byref(axes(**ax)), None) == want
    for kw, want in ((dict(theta=0.0), ERR_THETA), (dict(q=None), ERR_NULL), (dict(reserved=1), ERR_UNSUPPORTED)):
        assert lib.rope_kv_append_axes(ctypes.byref(append(**kw)), ctypes.byref(axes()), None) == want


def step(**kw):
    from packed_varlen_rope_gb300 import PagedKVStepDesc

    d = PagedKVStepDesc()
    for i, name in enumerate(("free_pages", "free_count", "count_out", "page_table", "past_lens", "new_lens", "finished",
                              "cu_seqlens", "kv_lens", "slots", "status")):
        setattr(d, name, BASE + (i << 30))
    d.page_table_stride, d.n_free_max, d.max_tokens, d.n_seqs, d.max_pages, d.page_size = 10, 100, 50, 4, 10, 16
    for k, v in kw.items():
        assert hasattr(d, k)
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,want", [
    (dict(n_seqs=-1), ERR_SHAPE), (dict(n_seqs=(1 << 24) + 1), ERR_SHAPE), (dict(max_pages=-1), ERR_SHAPE),
    (dict(page_size=0), ERR_SHAPE), (dict(page_size=65537), ERR_SHAPE), (dict(n_free_max=-1), ERR_SHAPE),
    (dict(n_free_max=1 << 31), ERR_SHAPE), (dict(max_tokens=-1), ERR_SHAPE), (dict(max_tokens=1 << 31), ERR_SHAPE),
    (dict(page_table_stride=9), ERR_SHAPE), (dict(reserved=1), ERR_UNSUPPORTED),
    (dict(max_pages=1 << 27, page_table_stride=1 << 27), ERR_UNSUPPORTED),
    (dict(max_pages=(1 << 24) + 1, page_table_stride=1 << 25, page_size=1), ERR_UNSUPPORTED),
    (dict(free_pages=None), ERR_NULL), (dict(free_count=None), ERR_NULL), (dict(count_out=None), ERR_NULL),
    (dict(page_table=None), ERR_NULL), (dict(past_lens=None), ERR_NULL), (dict(new_lens=None), ERR_NULL),
    (dict(cu_seqlens=None), ERR_NULL), (dict(kv_lens=None), ERR_NULL), (dict(slots=BASE + (9 << 30) + 4), ERR_ALIGN),
    (dict(past_lens=BASE + (4 << 30) + 2), ERR_ALIGN), (dict(kv_lens=BASE + (4 << 30)), ERR_OVERLAP),
    (dict(status=BASE + (1 << 30)), ERR_OVERLAP), (dict(count_out=BASE + (3 << 30) + 4), ERR_OVERLAP),
    (dict(cu_seqlens=BASE + (9 << 30)), ERR_OVERLAP), (dict(finished=BASE + (3 << 30)), ERR_OVERLAP),
    (dict(count_out=BASE + (1 << 30), status=BASE + (1 << 30)), ERR_OVERLAP),
])
def test_step_refusals(lib, kw, want):
    assert lib.paged_kv_step(ctypes.byref(step(**kw)), None) == want


def test_step_without_a_descriptor(lib):
    assert lib.paged_kv_step(None, None) == ERR_NULL


def test_tensors_of_the_host_are_refused():
    """Before the library is asked for anything."""
    import packed_varlen_rope_gb300 as m

    torch = pytest.importorskip("torch")
    i32 = torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        m.paged_kv_step(torch.arange(4, dtype=i32), torch.tensor([4], dtype=i32), torch.zeros((1, 2), dtype=i32),
                        torch.zeros(1, dtype=i32), torch.ones(1, dtype=i32), 8, 4)
    q, k, ids = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros((3, 1, 64), dtype=torch.bfloat16), torch.zeros((2, 3), dtype=i32)
    for call in (m.rope_axes_apply, m.apply_rope_axes):
        with pytest.raises(ValueError):
            call(q, k, 1e4, (16, 16), ids)
    with pytest.raises(ValueError):
        m.RotaryEmbedding(64, 1e4, use_cache=False, sections=(16, 16))(q, k, position_ids=ids)
    for kw in (dict(sections=(16, 15)), dict(sections=()), dict(sections=(8,) * 5), dict(interleaved=True), dict(own_frequencies=True)):
        with pytest.raises(ValueError):
            m.RotaryEmbedding(64, 1e4, **kw)
