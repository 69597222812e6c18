"""ctypes binding of the attention entry points and the paged cache (``include/attn.h``,
``include/paged_kv.h``): argument marshalling only, in the manner of ``_binding``."""
from __future__ import annotations

import ctypes
import math
from typing import Optional

from ._binding import (RopeCosSinCacheDesc, _cache_arg, _check, _check_cu, _on, _ptr, _stream, _view_args,
                       load_library)

ATTN_EXPORTS = ("attn_varlen_fwd", "attn_varlen_bwd", "attn_varlen_bwd_workspace_bytes", "attn_paged",
                "attn_paged_workspace_bytes", "attn_fault")

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


def _view_fields(name):
    return [(name, _vp), (name + "_stride_token", _i64), (name + "_stride_head", _i64)]


class RopePagedKV(ctypes.Structure):
    """Mirror of ``rope_paged_kv`` in include/paged_kv.h."""

    _fields_ = [("k", _vp), ("k_stride_page", _i64), ("k_stride_token", _i64), ("k_stride_head", _i64),
                ("v", _vp), ("v_stride_page", _i64), ("v_stride_token", _i64), ("v_stride_head", _i64),
                ("n_pages", _i64), ("page_size", _i32), ("n_kv_heads", _i32), ("head_dim", _i32),
                ("reserved", _i32)]


class RopeKVAppendDesc(ctypes.Structure):
    """Mirror of ``rope_kv_append_desc``."""

    _fields_ = [*_view_fields("q"), *_view_fields("k"), *_view_fields("v"), *_view_fields("q_out"),
                ("cache", RopePagedKV), ("cu_seqlens", _vp), ("kv_lens", _vp), ("page_table", _vp),
                ("page_table_stride", _i64), ("max_pages", _i32), ("n_seqs", _i32), ("n_q_heads", _i32),
                ("reserved", _i32), ("total_tokens", _i64), ("theta", ctypes.c_double),
                ("position_scale", ctypes.c_double), ("cos_sin_cache", ctypes.POINTER(RopeCosSinCacheDesc))]


class AttnVarlenDesc(ctypes.Structure):
    """Mirror of ``attn_varlen_desc`` in include/attn.h."""

    _fields_ = [*_view_fields("q"), *_view_fields("k"), *_view_fields("v"), *_view_fields("out"),
                ("lse", _vp), ("cu_seqlens", _vp), ("seq_used", _vp), ("total_tokens", _i64), ("n_seqs", _i32),
                ("n_q_heads", _i32), ("n_kv_heads", _i32), ("head_dim", _i32), ("causal", _i32),
                ("scale", ctypes.c_float)]


class AttnVarlenGrads(ctypes.Structure):
    """Mirror of ``attn_varlen_grads``."""

    _fields_ = [*_view_fields("dout"), *_view_fields("dq"), *_view_fields("dk"), *_view_fields("dv")]


class AttnPagedDesc(ctypes.Structure):
    """Mirror of ``attn_paged_desc``."""

    _fields_ = [*_view_fields("q"), *_view_fields("out"), ("cache", RopePagedKV), ("cu_seqlens", _vp),
                ("kv_lens", _vp), ("page_table", _vp), ("page_table_stride", _i64), ("total_tokens", _i64),
                ("max_kv_len", _i64), ("max_pages", _i32), ("n_seqs", _i32), ("n_q_heads", _i32),
                ("causal", _i32), ("scale", ctypes.c_float), ("reserved", _i32)]


def _declare(lib):
    """Signatures of the entry points (called by ``load_library``)."""
    p = ctypes.POINTER
    lib.rope_kv_append.argtypes = [p(RopeKVAppendDesc), _vp]
    lib.attn_varlen_fwd.argtypes = [p(AttnVarlenDesc), _vp]
    lib.attn_varlen_bwd.argtypes = [p(AttnVarlenDesc), p(AttnVarlenGrads), _vp, _i64, _vp]
    lib.attn_varlen_bwd_workspace_bytes.argtypes = [_i64, _i32]
    lib.attn_varlen_bwd_workspace_bytes.restype = _i64
    lib.attn_paged.argtypes = [p(AttnPagedDesc), _vp, _i64, _vp]
    lib.attn_paged_workspace_bytes.argtypes = [p(AttnPagedDesc)]
    lib.attn_paged_workspace_bytes.restype = _i64
    lib.attn_fault.argtypes = []
    for name in ("rope_kv_append", "attn_varlen_fwd", "attn_varlen_bwd", "attn_paged", "attn_fault"):
        getattr(lib, name).restype = ctypes.c_int


class PagedKVCache:
    """Keys and values in pages: ``k_pages`` and ``v_pages`` are bf16 CUDA views
    [n_pages, page_size, n_kv_heads, head_dim], head_dim contiguous, any other strides (the
    two may be the halves of one pool).  page_size is a multiple of 8."""

    def __init__(self, k_pages, v_pages):
        import torch

        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 4 or (t.numel() and t.stride(3) != 1):
                raise ValueError("%s must be a CUDA bf16 [pages, page_size, kv_heads, head_dim] view with head_dim "
                                 "contiguous" % name)
        if k_pages.shape != v_pages.shape or k_pages.device != v_pages.device:
            raise ValueError("k_pages and v_pages must share shape and device")
        self.k_pages, self.v_pages = k_pages, v_pages
        n, page, heads, d = k_pages.shape
        ks, vs = k_pages.stride(), v_pages.stride()
        self.desc = RopePagedKV(k_pages.data_ptr(), ks[0], ks[1], ks[2], v_pages.data_ptr(), vs[0], vs[1], vs[2],
                                n, page, heads, d, 0)

    @property
    def device(self):
        return self.k_pages.device

    @property
    def n_pages(self) -> int:
        return self.desc.n_pages

    @property
    def page_size(self) -> int:
        return self.desc.page_size

    @property
    def n_kv_heads(self) -> int:
        return self.desc.n_kv_heads

    @property
    def head_dim(self) -> int:
        return self.desc.head_dim


def new_paged_kv_cache(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda") -> PagedKVCache:
    """Allocate (through torch, uninitialised) the pages of one layer's cache."""
    import torch

    shape = (int(n_pages), int(page_size), int(n_kv_heads), int(head_dim))
    return PagedKVCache(torch.empty(shape, dtype=torch.bfloat16, device=device),
                        torch.empty(shape, dtype=torch.bfloat16, device=device))


def _tables(desc, cache, device, page_table, kv_lens, cu_seqlens):
    import torch

    if not isinstance(cache, PagedKVCache):
        raise ValueError("cache must be a PagedKVCache")
    if cache.device != device:
        raise ValueError("the cache is on %s, q on %s" % (cache.device, device))
    _check_cu(cu_seqlens, device)
    n = cu_seqlens.numel() - 1
    if n < 0:
        raise ValueError("cu_seqlens must hold n_seqs + 1 offsets")
    if kv_lens.dtype != torch.int32 or kv_lens.device != device or not kv_lens.is_contiguous() or kv_lens.numel() != n:
        raise ValueError("kv_lens must be a contiguous int32 tensor of one length per sequence on the device of q")
    if page_table.dtype != torch.int32 or page_table.device != device or page_table.dim() != 2 or \
            page_table.shape[0] != n or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be an int32 [n_seqs, max_pages] tensor with contiguous rows on the "
                         "device of q")
    desc.cache = cache.desc
    desc.cu_seqlens, desc.kv_lens, desc.page_table = _ptr(cu_seqlens), _ptr(kv_lens), _ptr(page_table)
    desc.page_table_stride, desc.max_pages, desc.n_seqs = page_table.stride(0), page_table.shape[1], n


def _keep_for(stream, *tensors):
    """Tensors allocated here, on torch's current stream, and used on ``stream``: their
    memory is not given to others before that stream has passed this point."""
    import torch

    if stream is None:
        return
    s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
    for t in tensors:
        if t is not None and t.numel():
            t.record_stream(s)


def _scale(scale, d: int) -> float:
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def rope_kv_append(q, k, v, cache: PagedKVCache, page_table, kv_lens, cu_seqlens, theta: float, q_out=None,
                   position_scale: float = 1.0, cos_sin_cache=None, stream=None):
    """Rotate the new tokens' q [T, Hq, d] (in place, or into ``q_out``) and k [T, Hkv, d] by
    their positions and write k and v [T, Hkv, d] into the pages of ``cache`` (C entry point
    ``rope_kv_append``).  ``cu_seqlens`` (int32 [n + 1]) delimits the new tokens of each
    sequence, ``kv_lens`` (int32 [n]) counts its tokens in the cache with the new ones,
    ``page_table`` (int32 [n, max_pages]) names its pages; all on the device.  k and v are
    only read.  Returns the rotated q."""
    desc = RopeKVAppendDesc()
    desc.q, desc.q_stride_token, desc.q_stride_head = _view_args(q, "q")
    desc.k, desc.k_stride_token, desc.k_stride_head = _view_args(k, "k")
    desc.v, desc.v_stride_token, desc.v_stride_head = _view_args(v, "v")
    T, hq, d = q.shape
    if k.shape != v.shape or k.shape[0] != T or k.shape[2] != d or k.device != q.device or v.device != q.device:
        raise ValueError("q, k and v must share tokens, head_dim and device, k and v their heads")
    _tables(desc, cache, q.device, page_table, kv_lens, cu_seqlens)
    if k.shape[1] != cache.n_kv_heads or d != cache.head_dim:
        raise ValueError("the cache holds %d heads of %d, k has %d of %d" % (cache.n_kv_heads, cache.head_dim,
                                                                            k.shape[1], d))
    if q_out is not None:
        if q_out.shape != q.shape or q_out.device != q.device:
            raise ValueError("q_out must have the shape and device of q")
        desc.q_out, desc.q_out_stride_token, desc.q_out_stride_head = _view_args(q_out, "q_out")
    desc.n_q_heads, desc.total_tokens = hq, T
    desc.theta, desc.position_scale = float(theta), float(position_scale)
    ref = _cache_arg(cos_sin_cache, d, q.device)
    if ref is not None:
        desc.cos_sin_cache = ref
    st = _on(q.device, load_library().rope_kv_append, ctypes.byref(desc), _stream(stream, q.device))
    _check("rope_kv_append", st)
    return q if q_out is None else q_out


def attn_paged(q, cache: PagedKVCache, page_table, kv_lens, cu_seqlens, causal: bool = True,
               scale: Optional[float] = None, out=None, max_kv_len: int = 0, workspace=None, stream=None):
    """Attention of the new tokens' q [T, Hq, d] over the pages of ``cache`` (C entry point
    ``attn_paged``), the new tokens' own keys and values among them (``rope_kv_append``
    first).  Arrays as for ``rope_kv_append``.  ``scale``: 1/sqrt(d) unless given.
    ``max_kv_len``: an upper bound on ``kv_lens`` known on the host (tunes the split of long
    caches; 0: what the page table's width allows).  ``workspace``: a CUDA tensor for
    partial results (``attn_paged_workspace_bytes``); allocated through torch unless given.
    Returns ``out`` [T, Hq, d] (a new tensor unless given)."""
    import torch

    desc = _paged_desc(q, cache, page_table, kv_lens, cu_seqlens, causal, scale, max_kv_len)
    made = out is None
    if made:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    elif out.shape != q.shape or out.device != q.device:
        raise ValueError("out must have the shape and device of q")
    desc.out, desc.out_stride_token, desc.out_stride_head = _view_args(out, "out")
    lib = load_library()
    own = None
    if workspace is None:
        need = int(lib.attn_paged_workspace_bytes(ctypes.byref(desc)))
        if need > 0:
            workspace = own = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif not workspace.is_cuda or workspace.device != q.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the device of q")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = _on(q.device, lib.attn_paged, ctypes.byref(desc), _ptr(workspace), nbytes, _stream(stream, q.device))
    _check("attn_paged", st)
    _keep_for(stream, own, out if made else None)
    return out


def _paged_desc(q, cache, page_table, kv_lens, cu_seqlens, causal, scale, max_kv_len):
    desc = AttnPagedDesc()
    desc.q, desc.q_stride_token, desc.q_stride_head = _view_args(q, "q")
    _tables(desc, cache, q.device, page_table, kv_lens, cu_seqlens)
    if q.shape[2] != cache.head_dim:
        raise ValueError("the cache holds heads of %d, q has %d" % (cache.head_dim, q.shape[2]))
    desc.total_tokens, desc.n_q_heads = q.shape[0], q.shape[1]
    desc.max_kv_len, desc.causal = int(max_kv_len), 1 if causal else 0
    desc.scale = _scale(scale, q.shape[2])
    return desc


def attn_paged_workspace_bytes(q, cache: PagedKVCache, page_table, kv_lens, cu_seqlens, max_kv_len: int = 0) -> int:
    """Bytes of workspace ``attn_paged`` needs for these arguments (0: none)."""
    desc = _paged_desc(q, cache, page_table, kv_lens, cu_seqlens, True, None, max_kv_len)
    need = int(load_library().attn_paged_workspace_bytes(ctypes.byref(desc)))
    if need < 0:
        _check("attn_paged_workspace_bytes", need)
    return need


def _varlen_desc(q, k, v, out, lse, cu_seqlens, causal, scale, seq_used):
    import torch

    desc = AttnVarlenDesc()
    desc.q, desc.q_stride_token, desc.q_stride_head = _view_args(q, "q")
    desc.k, desc.k_stride_token, desc.k_stride_head = _view_args(k, "k")
    desc.v, desc.v_stride_token, desc.v_stride_head = _view_args(v, "v")
    desc.out, desc.out_stride_token, desc.out_stride_head = _view_args(out, "out")
    T, hq, d = q.shape
    dev = q.device
    if k.shape != v.shape or k.shape[0] != T or k.shape[2] != d or k.device != dev or v.device != dev:
        raise ValueError("q, k and v must share tokens, head_dim and device, k and v their heads")
    if out.shape != q.shape or out.device != dev:
        raise ValueError("out must have the shape and device of q")
    if lse is not None:
        if lse.dtype != torch.float32 or lse.device != dev or tuple(lse.shape) != (hq, T) or not lse.is_contiguous():
            raise ValueError("lse must be a contiguous float32 [heads, tokens] tensor on the device of q")
        desc.lse = _ptr(lse)
    _check_cu(cu_seqlens, dev)
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold n_seqs + 1 offsets")
    desc.cu_seqlens, desc.n_seqs = _ptr(cu_seqlens), cu_seqlens.numel() - 1
    if seq_used is not None:
        _check_cu(seq_used, dev)
        if seq_used.numel() != desc.n_seqs:
            raise ValueError("seq_used must hold one int32 per sample")
        desc.seq_used = _ptr(seq_used)
    desc.total_tokens, desc.n_q_heads, desc.n_kv_heads, desc.head_dim = T, hq, k.shape[1], d
    desc.causal, desc.scale = 1 if causal else 0, _scale(scale, d)
    return desc


def attn_varlen_fwd(q, k, v, cu_seqlens, causal: bool = True, scale: Optional[float] = None, seq_used=None, out=None,
                    return_lse: bool = False, stream=None):
    """Attention within each sample of a pack (C entry point ``attn_varlen_fwd``).  q
    [T, Hq, d], k and v [T, Hkv, d]: bf16 CUDA views, any token and head strides (the
    slices of one fused QKV output), Hq a multiple of Hkv, d a multiple of 16 up to 128.
    ``seq_used`` (int32 [n]): only the first seq_used[s] rows of sample s are rows and keys.
    ``scale``: 1/sqrt(d) unless given.  Returns out [T, Hq, d] (a new tensor unless given;
    rows that see no key are 0), with ``return_lse`` (out, lse): lse float32 [Hq, T], the
    natural logarithm of each row's sum, which the backward takes."""
    import torch

    made = out is None
    if made:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device) if return_lse else None
    desc = _varlen_desc(q, k, v, out, lse, cu_seqlens, causal, scale, seq_used)
    st = _on(q.device, load_library().attn_varlen_fwd, ctypes.byref(desc), _stream(stream, q.device))
    _check("attn_varlen_fwd", st)
    _keep_for(stream, out if made else None, lse)
    return (out, lse) if return_lse else out


def attn_varlen_bwd(dout, q, k, v, out, lse, cu_seqlens, causal: bool = True, scale: Optional[float] = None,
                    seq_used=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of ``attn_varlen_fwd`` for the output gradient ``dout`` (C entry
    point ``attn_varlen_bwd``), with the ``out`` and ``lse`` that it returned and its other
    arguments.  dq, dk and dv are written whole (new tensors unless given; rows of no sample
    get 0).  ``workspace``: a CUDA tensor of at least 8 * T * Hq bytes; allocated through
    torch unless given."""
    import torch

    if lse is None:
        raise ValueError("the backward needs the forward's lse (return_lse=True)")
    desc = _varlen_desc(q, k, v, out, lse, cu_seqlens, causal, scale, seq_used)
    g = AttnVarlenGrads()
    made = []
    grads = []
    for name, t, like in (("dout", dout, q), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is None:
            if name == "dout":
                raise ValueError("dout is required")
            t = torch.empty(like.shape, dtype=torch.bfloat16, device=q.device)
            made.append(t)
        elif t.shape != like.shape or t.device != q.device:
            raise ValueError("%s must have shape %s on %s" % (name, tuple(like.shape), q.device))
        p, ts, hs = _view_args(t, name)
        setattr(g, name, p)
        setattr(g, name + "_stride_token", ts)
        setattr(g, name + "_stride_head", hs)
        grads.append(t)
    lib = load_library()
    if workspace is None:
        need = int(lib.attn_varlen_bwd_workspace_bytes(q.shape[0], q.shape[1]))
        workspace = torch.empty(max(need, 0), dtype=torch.uint8, device=q.device)
        made.append(workspace)
    elif not workspace.is_cuda or workspace.device != q.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the device of q")
    st = _on(q.device, lib.attn_varlen_bwd, ctypes.byref(desc), ctypes.byref(g), _ptr(workspace),
             workspace.numel() * workspace.element_size(), _stream(stream, q.device))
    _check("attn_varlen_bwd", st)
    _keep_for(stream, *made)
    return tuple(grads[1:])


def attn_fault() -> bool:
    """Whether a bounded wait inside an attention kernel has run out on the current device
    since the library was loaded.  Synchronises the device."""
    return load_library().attn_fault() != 0


_Attn = None


def _attn_function():
    import torch

    class Attn(torch.autograd.Function):
        """Autograd wrapper of the packed attention: q, k, v, out and lse are saved."""

        @staticmethod
        def forward(ctx, q, k, v, cu_seqlens, causal, scale, seq_used):
            out, lse = attn_varlen_fwd(q, k, v, cu_seqlens, causal, scale, seq_used, return_lse=True)
            ctx.save_for_backward(q, k, v, out, lse, cu_seqlens, seq_used)
            ctx.args = (causal, scale)
            return out

        @staticmethod
        def backward(ctx, dout):
            q, k, v, out, lse, cu_seqlens, seq_used = ctx.saved_tensors
            dq, dk, dv = attn_varlen_bwd(_rows(dout), q, k, v, out, lse, cu_seqlens, *ctx.args, seq_used=seq_used)
            return dq, dk, dv, None, None, None, None

    return Attn


def _rows(t):
    """``t`` itself when the kernels can address it, else a contiguous copy (a broadcast
    tensor: stride 0; a head_dim that is not contiguous; odd strides or an odd start)."""
    ok = t.dim() == 3 and t.stride(2) == 1 and t.data_ptr() % 16 == 0 and \
        all(t.stride(i) % 8 == 0 and (t.stride(i) > 0 or t.shape[i] == 1) for i in (0, 1))
    return t if ok else t.clone(memory_format=__import__("torch").contiguous_format)


def apply_attn(q, k, v, cu_seqlens, causal: bool = True, scale: Optional[float] = None, seq_used=None):
    """Differentiable attention within each sample of a pack: ``attn_varlen_fwd`` with the
    gradients of ``attn_varlen_bwd``.  q, k, v may be any bf16 CUDA [T, heads, d] tensors;
    those that the kernels cannot address (broadcast ones) are copied."""
    global _Attn
    if _Attn is None:
        _Attn = _attn_function()
    return _Attn.apply(_rows(q), _rows(k), _rows(v), cu_seqlens, bool(causal), scale, seq_used)
