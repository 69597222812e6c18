"""The attention entry points' host side (no GPU): declarations against exports, the binding's
structures and packed descriptors against the C compiler's layout, and every refusal that is
made before anything is launched."""
from __future__ import annotations

import ctypes
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INCLUDE = os.path.join(ROOT, "include")

OK, ERR_NULL, ERR_SHAPE, ERR_HEAD_DIM, ERR_ALIGN, ERR_OVERLAP, ERR_UNSUPPORTED, ERR_LAUNCH, ERR_THETA = \
    0, -1, -2, -3, -4, -5, -6, -7, -8
ERR_WORKSPACE, ERR_CACHE = -10, -11


@pytest.fixture(scope="module")
def lib():
    from packed_varlen_rope_gb300 import build, load_library

    build.build()
    return load_library()


def test_attention_exports_match_the_header(lib):
    from packed_varlen_rope_gb300 import ATTN_EXPORTS

    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, "attn.h")).read(), flags=re.S)
    declared = re.findall(r"^\s*(?:int|int64_t)\s+(attn_\w+)\s*\(", text, flags=re.M)
    assert sorted(ATTN_EXPORTS) == sorted(declared)
    assert all(hasattr(lib, n) for n in declared)


def test_headers_are_plain_c_and_structures_match(tmp_path):
    """Size and every field's offset of the binding's structures, as gcc lays them out; the
    packed formats have the same sizes."""
    from packed_varlen_rope_gb300 import _attention as A

    pairs = (("rope_paged_kv", A.RopePagedKV), ("rope_kv_append_desc", A.RopeKVAppendDesc),
             ("attn_varlen_desc", A.AttnVarlenDesc), ("attn_varlen_grads", A.AttnVarlenGrads),
             ("attn_paged_desc", A.AttnPagedDesc))
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "attn.h"', "int main(void) {"]
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
    for pack, st in ((A._KV_PACK, A.RopePagedKV), (A._APPEND_PACK, A.RopeKVAppendDesc), (A._VARLEN_PACK, A.AttnVarlenDesc),
                     (A._GRADS_PACK, A.AttnVarlenGrads), (A._PAGED_PACK, A.AttnPagedDesc)):
        assert pack.__self__.size == ctypes.sizeof(st)


def test_packed_descriptor_fills_the_fields_in_order():
    from packed_varlen_rope_gb300 import _attention as A

    kv = A._KV_PACK(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 0)
    d = A.AttnPagedDesc.from_buffer_copy(A._PAGED_PACK(21, 22, 23, 24, 25, 26, kv, 31, 32, 33, 34, 35, 36, 37, 38, 39,
                                                       1, 0.5, 0))
    assert (d.q, d.q_stride_token, d.q_stride_head, d.out, d.out_stride_token, d.out_stride_head) == tuple(range(21, 27))
    c = d.cache
    assert (c.k, c.k_stride_page, c.k_stride_token, c.k_stride_head, c.v, c.v_stride_page, c.v_stride_token,
            c.v_stride_head, c.n_pages, c.page_size, c.n_kv_heads, c.head_dim, c.reserved) == (*range(1, 13), 0)
    assert (d.cu_seqlens, d.kv_lens, d.page_table, d.page_table_stride, d.total_tokens, d.max_kv_len, d.max_pages,
            d.n_seqs, d.n_q_heads, d.causal, d.scale, d.reserved) == (*range(31, 40), 1, 0.5, 0)
    v = A.AttnVarlenDesc.from_buffer_copy(A._VARLEN_PACK(*range(1, 13), 13, 14, 15, 16, 17, 18, 19, 20, 1, 0.25))
    assert (v.lse, v.cu_seqlens, v.seq_used, v.total_tokens, v.n_seqs, v.n_q_heads, v.n_kv_heads, v.head_dim, v.causal,
            v.scale) == (*range(13, 21), 1, 0.25)
    a = A.RopeKVAppendDesc.from_buffer_copy(A._APPEND_PACK(*range(1, 13), kv, 14, 15, 16, 17, 18, 19, 20, 0, 21, 1e6, 2.0, 0))
    assert (a.cu_seqlens, a.kv_lens, a.page_table, a.page_table_stride, a.max_pages, a.n_seqs, a.n_q_heads,
            a.total_tokens, a.theta, a.position_scale, bool(a.cos_sin_cache)) == (*range(14, 22), 1e6, 2.0, False)


# Pointers below are made up: every call here is refused before any is followed.
BASE = 1 << 40


def varlen(**kw):
    from packed_varlen_rope_gb300 import AttnVarlenDesc

    T, hq, hkv, d = kw.pop("T", 100), kw.pop("hq", 8), kw.pop("hkv", 2), kw.pop("d", 64)
    a = AttnVarlenDesc()
    at = BASE
    for name, h in (("q", hq), ("k", hkv), ("v", hkv), ("out", hq)):
        setattr(a, name, at)
        setattr(a, name + "_stride_token", h * d)
        setattr(a, name + "_stride_head", d)
        at += 1 << 30
    a.lse, a.cu_seqlens = at, at + (1 << 24)
    a.total_tokens, a.n_seqs, a.n_q_heads, a.n_kv_heads, a.head_dim, a.causal, a.scale = T, 1, hq, hkv, d, 1, 0.125
    for k, v in kw.items():
        assert hasattr(a, k), k
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(total_tokens=-1), ERR_SHAPE), (dict(n_seqs=-1), ERR_SHAPE), (dict(n_q_heads=0), ERR_SHAPE),
    (dict(n_kv_heads=0), ERR_SHAPE), (dict(n_kv_heads=3), ERR_SHAPE), (dict(n_seqs=(1 << 24) + 1), ERR_SHAPE),
    (dict(head_dim=0), ERR_HEAD_DIM), (dict(head_dim=8), ERR_HEAD_DIM), (dict(head_dim=72), ERR_HEAD_DIM),
    (dict(head_dim=144), ERR_HEAD_DIM), (dict(head_dim=256), ERR_HEAD_DIM),
    (dict(n_q_heads=129, n_kv_heads=1), ERR_UNSUPPORTED), (dict(total_tokens=(1 << 24) + 1), ERR_UNSUPPORTED),
    (dict(total_tokens=1 << 24, n_q_heads=128, n_kv_heads=2), ERR_UNSUPPORTED),
    (dict(scale=0.0), ERR_THETA), (dict(scale=-1.0), ERR_THETA), (dict(scale=float("nan")), ERR_THETA),
    (dict(scale=float("inf")), ERR_THETA),
    (dict(q=None), ERR_NULL), (dict(k=None), ERR_NULL), (dict(v=None), ERR_NULL), (dict(out=None), ERR_NULL),
    (dict(cu_seqlens=None), ERR_NULL), (dict(q=BASE + 8), ERR_ALIGN), (dict(v_stride_token=132), ERR_ALIGN),
    (dict(k_stride_head=-64), ERR_SHAPE), (dict(q_stride_token=0), ERR_OVERLAP), (dict(k_stride_head=0), ERR_OVERLAP),
    (dict(out=BASE), ERR_OVERLAP), (dict(out=BASE + (1 << 30)), ERR_OVERLAP), (dict(lse=BASE + 2), ERR_ALIGN),
])
def test_varlen_refusals(lib, kw, want):
    assert lib.attn_varlen_fwd(ctypes.byref(varlen(**kw)), None) == want


def grads(T=100, hq=8, hkv=2, d=64, **kw):
    from packed_varlen_rope_gb300 import AttnVarlenGrads

    g = AttnVarlenGrads()
    at = BASE + (1 << 36)
    for name, h in (("dout", hq), ("dq", hq), ("dk", hkv), ("dv", hkv)):
        setattr(g, name, at)
        setattr(g, name + "_stride_token", h * d)
        setattr(g, name + "_stride_head", d)
        at += 1 << 30
    for k, v in kw.items():
        setattr(g, k, v)
    return g


@pytest.mark.parametrize("kw,gw,ws,nbytes,want", [
    (dict(lse=None), {}, BASE, 1 << 20, ERR_NULL), ({}, dict(dout=None), BASE, 1 << 20, ERR_NULL),
    ({}, dict(dk=None), BASE, 1 << 20, ERR_NULL), ({}, {}, None, 1 << 20, ERR_NULL),
    ({}, {}, BASE + 8, 1 << 20, ERR_ALIGN), ({}, {}, BASE, 100 * 8 * 8 - 1, ERR_WORKSPACE),
    ({}, dict(dq=BASE), BASE, 1 << 20, ERR_OVERLAP), ({}, dict(dk=BASE + (1 << 36)), BASE, 1 << 20, ERR_OVERLAP),
    ({}, dict(dv=BASE + (1 << 36) + (2 << 30)), BASE, 1 << 20, ERR_OVERLAP),
    ({}, dict(dv_stride_head=4), BASE, 1 << 20, ERR_ALIGN), (dict(head_dim=24), {}, BASE, 1 << 20, ERR_HEAD_DIM),
])
def test_backward_refusals(lib, kw, gw, ws, nbytes, want):
    assert lib.attn_varlen_bwd(ctypes.byref(varlen(**kw)), ctypes.byref(grads(**gw)), ws, nbytes, None) == want


def test_backward_workspace_size(lib):
    f = lib.attn_varlen_bwd_workspace_bytes
    assert f(100, 8) == 100 * 8 * 8 and f(0, 8) == 0
    assert f(-1, 8) == -1 and f(100, 0) == -1 and f((1 << 24) + 1, 1) == -1


def test_nothing_to_do_reads_no_pointer(lib):
    from packed_varlen_rope_gb300 import AttnPagedDesc, AttnVarlenDesc, RopeKVAppendDesc

    d = AttnVarlenDesc()
    d.n_q_heads, d.n_kv_heads, d.head_dim, d.scale = 8, 2, 64, 1.0
    assert lib.attn_varlen_fwd(ctypes.byref(d), None) == OK
    assert lib.attn_varlen_bwd(ctypes.byref(d), ctypes.byref(grads()), None, 0, None) == OK
    p = AttnPagedDesc()
    p.n_q_heads, p.scale = 8, 1.0
    p.cache.n_kv_heads, p.cache.head_dim, p.cache.page_size = 2, 64, 16
    assert lib.attn_paged(ctypes.byref(p), None, 0, None) == OK
    assert lib.attn_paged_workspace_bytes(ctypes.byref(p)) == 0
    a = RopeKVAppendDesc()
    a.n_q_heads, a.theta, a.position_scale = 8, 1e4, 1.0
    a.cache = p.cache
    assert lib.rope_kv_append(ctypes.byref(a), None) == OK
    for fn in (lib.attn_varlen_fwd, lib.rope_kv_append):
        assert fn(None, None) == ERR_NULL
    assert lib.attn_paged(None, None, 0, None) == ERR_NULL


def kv_cache(c, pages=50, page=16, heads=2, d=64, **kw):
    c.k, c.v = BASE + (1 << 36), BASE + (1 << 37)
    for n in "kv":
        setattr(c, n + "_stride_page", page * heads * d)
        setattr(c, n + "_stride_token", heads * d)
        setattr(c, n + "_stride_head", d)
    c.n_pages, c.page_size, c.n_kv_heads, c.head_dim = pages, page, heads, d
    for k, v in kw.items():
        assert hasattr(c, k), k
        setattr(c, k, v)


def paged(cache=None, T=4, hq=8, d=64, **kw):
    from packed_varlen_rope_gb300 import AttnPagedDesc

    p = AttnPagedDesc()
    p.q, p.q_stride_token, p.q_stride_head = BASE, hq * d, d
    p.out, p.out_stride_token, p.out_stride_head = BASE + (1 << 30), hq * d, d
    kv_cache(p.cache, **(cache or {}))
    p.cu_seqlens, p.kv_lens, p.page_table = BASE + (2 << 30), BASE + (3 << 30), BASE + (4 << 30)
    p.page_table_stride, p.total_tokens, p.max_pages, p.n_seqs, p.n_q_heads, p.causal, p.scale = 10, T, 10, 4, hq, 1, 0.1
    for k, v in kw.items():
        assert hasattr(p, k), k
        setattr(p, k, v)
    return p


CACHE_REFUSALS = [
    (dict(n_pages=-1), ERR_SHAPE), (dict(page_size=0), ERR_SHAPE), (dict(page_size=12), ERR_SHAPE),
    (dict(page_size=1 << 17), ERR_SHAPE), (dict(reserved=1), ERR_UNSUPPORTED), (dict(k=None), ERR_NULL),
    (dict(v=None), ERR_NULL), (dict(k=BASE + (1 << 36) + 2), ERR_ALIGN), (dict(v_stride_token=132), ERR_ALIGN),
    (dict(k_stride_page=-64), ERR_SHAPE), (dict(k_stride_page=0), ERR_OVERLAP), (dict(v_stride_token=64), ERR_OVERLAP),
    (dict(v=BASE + (1 << 36)), ERR_OVERLAP), (dict(v=BASE + (1 << 36) + 16 * 2 * 64 * 2), ERR_OVERLAP),
]


@pytest.mark.parametrize("cache,want", CACHE_REFUSALS)
def test_cache_refusals(lib, cache, want):
    assert lib.attn_paged(ctypes.byref(paged(cache)), None, 1 << 30, None) == want
    assert lib.rope_kv_append(ctypes.byref(append(cache)), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(total_tokens=-1), ERR_SHAPE), (dict(n_q_heads=7), ERR_SHAPE), (dict(max_pages=-1), ERR_SHAPE),
    (dict(max_kv_len=-1), ERR_SHAPE), (dict(reserved=1), ERR_UNSUPPORTED), (dict(scale=0.0), ERR_THETA),
    (dict(page_table_stride=9), ERR_SHAPE), (dict(kv_lens=None), ERR_NULL), (dict(page_table=None), ERR_NULL),
    (dict(cu_seqlens=None), ERR_NULL), (dict(q=None), ERR_NULL), (dict(out=BASE), ERR_OVERLAP),
    (dict(out=BASE + (1 << 36)), ERR_OVERLAP), (dict(out=BASE + (1 << 30) + 4), ERR_ALIGN),
    (dict(max_pages=1 << 28, page_table_stride=1 << 28), ERR_UNSUPPORTED),
])
def test_paged_refusals(lib, kw, want):
    assert lib.attn_paged(ctypes.byref(paged(**kw)), None, 1 << 30, None) == want


def test_more_tiles_than_a_launch_counts(lib):
    """Tile slots times heads past 2^31: every sequence, empty or not, adds a slot."""
    ref, n = ctypes.byref, 1 << 24
    a = varlen(hq=256, hkv=256, n_seqs=n)
    assert lib.attn_varlen_fwd(ref(a), None) == ERR_UNSUPPORTED
    assert lib.attn_varlen_bwd(ref(a), ref(grads(hq=256, hkv=256)), BASE + (1 << 38), 1 << 20, None) == ERR_UNSUPPORTED
    p = paged(dict(heads=256), hq=256, n_seqs=n)
    assert lib.attn_paged(ref(p), BASE + (1 << 38), 1 << 40, None) == ERR_UNSUPPORTED
    assert lib.attn_paged_workspace_bytes(ref(p)) == ERR_UNSUPPORTED


def test_paged_head_dims(lib):
    """The cache holds head_dim up to 256; attention takes up to 128."""
    for d, want in ((144, ERR_HEAD_DIM), (256, ERR_HEAD_DIM), (20, ERR_HEAD_DIM)):
        assert lib.attn_paged(ctypes.byref(paged(dict(head_dim=d))), None, 1 << 30, None) == want


def test_paged_workspace(lib):
    """A split needs a workspace, as large as it says, aligned; the sizes alone decide."""
    p = paged(dict(pages=70000), T=1, hq=2, n_seqs=1, max_pages=65536, page_table_stride=65536)
    p.cache.n_kv_heads = 1
    need = lib.attn_paged_workspace_bytes(ctypes.byref(p))
    assert need > 0 and need % 4 == 0
    assert lib.attn_paged(ctypes.byref(p), None, need, None) == ERR_NULL
    assert lib.attn_paged(ctypes.byref(p), BASE + 4, need, None) == ERR_ALIGN
    assert lib.attn_paged(ctypes.byref(p), BASE + (5 << 30), need - 1, None) == ERR_WORKSPACE
    p.max_kv_len = 100
    assert lib.attn_paged_workspace_bytes(ctypes.byref(p)) == 0
    p.scale = -1.0
    assert lib.attn_paged_workspace_bytes(ctypes.byref(p)) == ERR_THETA
    assert lib.attn_paged_workspace_bytes(None) == ERR_NULL


def append(cache=None, T=4, hq=8, hkv=2, d=64, **kw):
    from packed_varlen_rope_gb300 import RopeKVAppendDesc

    a = RopeKVAppendDesc()
    at = BASE
    for name, h in (("q", hq), ("k", hkv), ("v", hkv), ("q_out", hq)):
        setattr(a, name, at)
        setattr(a, name + "_stride_token", h * d)
        setattr(a, name + "_stride_head", d)
        at += 1 << 30
    kv_cache(a.cache, **(cache or {}))
    a.cu_seqlens, a.kv_lens, a.page_table = BASE + (5 << 30), BASE + (6 << 30), BASE + (7 << 30)
    a.page_table_stride, a.max_pages, a.n_seqs, a.n_q_heads, a.total_tokens = 10, 10, 4, hq, T
    a.theta, a.position_scale = 1e4, 1.0
    for k, v in kw.items():
        assert hasattr(a, k), k
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(total_tokens=-1), ERR_SHAPE), (dict(n_q_heads=0), ERR_SHAPE), (dict(n_seqs=-1), ERR_SHAPE),
    (dict(reserved=1), ERR_UNSUPPORTED), (dict(total_tokens=(1 << 24) + 1), ERR_UNSUPPORTED),
    (dict(theta=0.0), ERR_THETA), (dict(theta=float("inf")), ERR_THETA), (dict(position_scale=-1.0), ERR_THETA),
    (dict(q=None), ERR_NULL), (dict(k=None), ERR_NULL), (dict(v=None), ERR_NULL), (dict(kv_lens=None), ERR_NULL),
    (dict(page_table=None), ERR_NULL), (dict(cu_seqlens=None), ERR_NULL), (dict(page_table_stride=3), ERR_SHAPE),
    (dict(q=BASE + 2), ERR_ALIGN), (dict(k_stride_token=20), ERR_ALIGN), (dict(v_stride_head=0), ERR_OVERLAP),
    (dict(q_out=BASE), ERR_OVERLAP), (dict(q_out=BASE + (2 << 30)), ERR_OVERLAP),
    (dict(q_out=None, k=BASE), ERR_OVERLAP), (dict(q=BASE + (1 << 36)), ERR_OVERLAP),
    (dict(q_out=BASE + (1 << 37)), ERR_OVERLAP),
])
def test_append_refusals(lib, kw, want):
    assert lib.rope_kv_append(ctypes.byref(append(**kw)), None) == want


def test_append_refuses_a_cache_descriptor_that_was_not_built(lib):
    from packed_varlen_rope_gb300 import RopeCosSinCacheDesc

    cs = RopeCosSinCacheDesc()
    cs.data, cs.rows, cs.head_dim, cs.theta, cs.position_scale = BASE, 10, 64, 1e4, 1.0
    a = append()
    a.cos_sin_cache = ctypes.pointer(cs)
    assert lib.rope_kv_append(ctypes.byref(a), None) == ERR_CACHE


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    import packed_varlen_rope_gb300 as pr

    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    pages = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: pr.attn_varlen_fwd(x, x, x, cu), lambda: pr.attn_varlen_bwd(x, x, x, x, x, None, cu),
                 lambda: pr.PagedKVCache(pages, pages), lambda: pr.apply_attn(x, x, x, cu)):
        with pytest.raises(ValueError):
            call()


def test_struct_formats_are_native():
    """The formats rely on native alignment, as the C compiler's."""
    assert struct.calcsize("@Pqi") == 24 - 4 and struct.calcsize("@P") == ctypes.sizeof(ctypes.c_void_p)
