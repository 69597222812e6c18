"""ctypes binding of the attention entry points and the paged cache (``include/attn.h``,
``include/paged_kv.h``): argument marshalling only, in the manner of ``_binding``."""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

from ._binding import RopeCosSinCacheDesc, _cache_arg, _check, _empty, load_library

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


# A decoding step is a few microseconds on the GPU, so the calls below pack a descriptor in one
# go (the structures above, as ``struct`` formats) and read each tensor's fields once.
_VIEW = "Pqq"
_KV_PACK = struct.Struct("@PqqqPqqqqiiii").pack
_PAGED = "88s"
_APPEND_PACK = struct.Struct("@" + 4 * _VIEW + _PAGED + "PPPqiiiiqddP").pack
_VARLEN_PACK = struct.Struct("@" + 4 * _VIEW + "PPPqiiiiif").pack
_GRADS_PACK = struct.Struct("@" + 4 * _VIEW).pack
_PAGED_PACK = struct.Struct("@" + 2 * _VIEW + _PAGED + "PPPqqqiiiifi").pack

_torch = _bf16 = _i32t = _f32t = _raw_stream = _current_device = None


def _load_torch():
    """torch, imported at the first call, and what every call needs of it."""
    global _torch, _bf16, _i32t, _f32t, _raw_stream, _current_device
    import torch

    _bf16, _i32t, _f32t = torch.bfloat16, torch.int32, torch.float32
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _current_device = getattr(torch._C, "_cuda_getDevice", None)
    _torch = torch
    return torch


def _view(t, name: str):
    """(pointer, token stride, head stride) of a bf16 CUDA [tokens, heads, head_dim] view."""
    st = t.stride()
    if len(st) != 3 or st[2] != 1 or t.dtype is not _bf16 or not t.is_cuda:
        raise ValueError("%s must be a CUDA bf16 [tokens, heads, head_dim] view with head_dim contiguous" % name)
    return t.data_ptr(), st[0], st[1]


def _int32(t, dev: int, n: int, what: str) -> int:
    """Pointer of a contiguous int32 [n] tensor on CUDA device ``dev``."""
    if t.dtype is not _i32t or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of %d values on the device of q" % (what, n))
    return t.data_ptr()


def _launch(fn, name: str, dev: int, stream, *args) -> None:
    """Call an entry point with device ``dev`` current, on ``stream`` (a torch stream or an int)
    or torch's current one of that device."""
    if stream is None:
        stream = _raw_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _current_device() == dev:
        st = fn(*args, stream)
    else:
        with _torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != 0:
        _check(name, st)


def _declare(lib):
    """Signatures of the entry points (called by ``load_library``).  Descriptors go as ``byref``
    of the structures above, or packed as bytes."""
    lib.rope_kv_append.argtypes = [_vp, _vp]
    lib.attn_varlen_fwd.argtypes = [_vp, _vp]
    lib.attn_varlen_bwd.argtypes = [_vp, _vp, _vp, _i64, _vp]
    lib.attn_varlen_bwd_workspace_bytes.argtypes = [_i64, _i32]
    lib.attn_varlen_bwd_workspace_bytes.restype = _i64
    lib.attn_paged.argtypes = [_vp, _vp, _i64, _vp]
    lib.attn_paged_workspace_bytes.argtypes = [_vp]
    lib.attn_paged_workspace_bytes.restype = _i64
    lib.attn_fault.argtypes = []
    for name in ("rope_kv_append", "attn_varlen_fwd", "attn_varlen_bwd", "attn_paged", "attn_fault"):
        getattr(lib, name).restype = ctypes.c_int


class PagedKVCache:
    """Keys and values in pages: ``k_pages`` and ``v_pages`` are bf16 CUDA views
    [n_pages, page_size, n_kv_heads, head_dim], head_dim contiguous, any other strides (the
    two may be the halves of one pool).  page_size is a multiple of 8.  Other pages are another
    PagedKVCache: the descriptor that the calls use holds these tensors' addresses."""

    def __init__(self, k_pages, v_pages):
        _torch or _load_torch()
        ks, vs, shape = k_pages.stride(), v_pages.stride(), k_pages.shape
        if k_pages.dtype is not _bf16 or v_pages.dtype is not _bf16 or not k_pages.is_cuda or len(ks) != 4 or \
                len(vs) != 4 or ((ks[3] != 1 or vs[3] != 1) and k_pages.numel()):
            raise ValueError("k_pages and v_pages must be CUDA bf16 [pages, page_size, kv_heads, head_dim] views with "
                             "head_dim contiguous")
        dev = k_pages.get_device()
        if shape != v_pages.shape or dev != v_pages.get_device():
            raise ValueError("k_pages and v_pages must share shape and device")
        self._k_pages, self._v_pages = k_pages, v_pages
        self._packed = _KV_PACK(k_pages.data_ptr(), ks[0], ks[1], ks[2], v_pages.data_ptr(), vs[0], vs[1], vs[2],
                                *shape, 0)
        self._dev, self._heads, self._dim = dev, shape[2], shape[3]

    @property
    def k_pages(self):
        return self._k_pages

    @property
    def v_pages(self):
        return self._v_pages

    @property
    def device(self):
        return self._k_pages.device

    @property
    def n_pages(self) -> int:
        return self._k_pages.shape[0]

    @property
    def page_size(self) -> int:
        return self._k_pages.shape[1]

    @property
    def n_kv_heads(self) -> int:
        return self._heads

    @property
    def head_dim(self) -> int:
        return self._dim

    @property
    def desc(self) -> RopePagedKV:
        """The C descriptor."""
        return RopePagedKV.from_buffer_copy(self._packed)


def new_paged_kv_cache(n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, device="cuda") -> PagedKVCache:
    """Allocate (through torch, uninitialised) the pages of one layer's cache."""
    import torch

    shape = (int(n_pages), int(page_size), int(n_kv_heads), int(head_dim))
    return PagedKVCache(torch.empty(shape, dtype=torch.bfloat16, device=device),
                        torch.empty(shape, dtype=torch.bfloat16, device=device))


def _tables(cache, dev: int, page_table, kv_lens, cu_seqlens):
    """The pointers and sizes (cu_seqlens, kv_lens, page_table, row stride, max_pages, n_seqs)."""
    if type(cache) is not PagedKVCache and not isinstance(cache, PagedKVCache):
        raise ValueError("cache must be a PagedKVCache")
    if cache._dev != dev:
        raise ValueError("the cache is on %s, q on cuda:%d" % (cache.device, dev))
    n = cu_seqlens.numel() - 1
    if n < 0:
        raise ValueError("cu_seqlens must hold n_seqs + 1 offsets")
    cu = _int32(cu_seqlens, dev, n + 1, "cu_seqlens")
    kv = _int32(kv_lens, dev, n, "kv_lens")
    st, shape = page_table.stride(), page_table.shape
    if page_table.dtype is not _i32t or page_table.get_device() != dev or len(st) != 2 or shape[0] != n or \
            (st[1] != 1 and shape[1] > 1):
        raise ValueError("page_table must be an int32 [n_seqs, max_pages] tensor with contiguous rows on the "
                         "device of q")
    return cu, kv, page_table.data_ptr(), st[0], shape[1], n


def rope_kv_append(q, k, v, cache: PagedKVCache, page_table, kv_lens, cu_seqlens, theta: float, q_out=None,
                   position_scale: float = 1.0, cos_sin_cache=None, stream=None):
    """Rotate the new tokens' q [T, Hq, d] (in place, or into ``q_out``) and k [T, Hkv, d] by
    their positions and write k and v [T, Hkv, d] into the pages of ``cache`` (C entry point
    ``rope_kv_append``).  ``cu_seqlens`` (int32 [n + 1]) delimits the new tokens of each
    sequence, ``kv_lens`` (int32 [n]) counts its tokens in the cache with the new ones,
    ``page_table`` (int32 [n, max_pages]) names its pages; all on the device.  k and v are
    only read.  Returns the rotated q."""
    _torch or _load_torch()
    qv, kv, vv = _view(q, "q"), _view(k, "k"), _view(v, "v")
    dev = q.get_device()
    T, hq, d = q.shape
    shape = k.shape
    if shape != v.shape or shape[0] != T or shape[2] != d or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k and v must share tokens, head_dim and device, k and v their heads")
    cu, lens, table, stride, width, n = _tables(cache, dev, page_table, kv_lens, cu_seqlens)
    if shape[1] != cache._heads or d != cache._dim:
        raise ValueError("the cache holds %d heads of %d, k has %d of %d" % (cache._heads, cache._dim, shape[1], d))
    ov = (0, 0, 0)
    if q_out is not None:
        if q_out.shape != q.shape or q_out.get_device() != dev:
            raise ValueError("q_out must have the shape and device of q")
        ov = _view(q_out, "q_out")
    ref = None
    if cos_sin_cache is not None:
        ref = _cache_arg(cos_sin_cache, d, q.device)
    desc = _APPEND_PACK(*qv, *kv, *vv, *ov, cache._packed, cu, lens, table, stride, width, n, hq, 0, T, float(theta),
                        float(position_scale), 0 if ref is None else ctypes.addressof(ref.contents))
    _launch(load_library().rope_kv_append, "rope_kv_append", dev, stream, desc)
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
    _torch or _load_torch()
    if out is None:
        out = _empty(q.shape, _bf16, q.device, stream)
    elif out.shape != q.shape or out.get_device() != q.get_device():
        raise ValueError("out must have the shape and device of q")
    desc, dev = _paged_desc(q, out, cache, page_table, kv_lens, cu_seqlens, causal, scale, max_kv_len)
    lib = load_library()
    if workspace is None:
        nbytes = lib.attn_paged_workspace_bytes(desc)
        if nbytes > 0:
            workspace = _empty(nbytes, _torch.uint8, q.device, stream, returned=False)
        ws = None if workspace is None else workspace.data_ptr()
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on the device of q")
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch(lib.attn_paged, "attn_paged", dev, stream, desc, ws, nbytes)
    return out


def _paged_desc(q, out, cache, page_table, kv_lens, cu_seqlens, causal, scale, max_kv_len):
    qv = _view(q, "q")
    ov = (0, 0, 0) if out is None else _view(out, "out")
    dev = q.get_device()
    T, hq, d = q.shape
    cu, lens, table, stride, width, n = _tables(cache, dev, page_table, kv_lens, cu_seqlens)
    if d != cache._dim:
        raise ValueError("the cache holds heads of %d, q has %d" % (cache._dim, d))
    return _PAGED_PACK(*qv, *ov, cache._packed, cu, lens, table, stride, T, int(max_kv_len), width, n, hq,
                       1 if causal else 0, d ** -0.5 if scale is None else scale, 0), dev


def attn_paged_workspace_bytes(q, cache: PagedKVCache, page_table, kv_lens, cu_seqlens, max_kv_len: int = 0) -> int:
    """Bytes of workspace ``attn_paged`` needs for these arguments (0: none)."""
    _torch or _load_torch()
    desc, _ = _paged_desc(q, None, cache, page_table, kv_lens, cu_seqlens, True, None, max_kv_len)
    need = int(load_library().attn_paged_workspace_bytes(desc))
    if need < 0:
        _check("attn_paged_workspace_bytes", need)
    return need


def _varlen_desc(q, k, v, out, lse, cu_seqlens, causal, scale, seq_used):
    """The packed descriptor, and the device."""
    qv, kv, vv, ov = _view(q, "q"), _view(k, "k"), _view(v, "v"), _view(out, "out")
    T, hq, d = q.shape
    dev = q.get_device()
    shape = k.shape
    if shape != v.shape or shape[0] != T or shape[2] != d or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k and v must share tokens, head_dim and device, k and v their heads")
    if out.shape != q.shape or out.get_device() != dev:
        raise ValueError("out must have the shape and device of q")
    lp = 0
    if lse is not None:
        if lse.dtype is not _f32t or lse.get_device() != dev or tuple(lse.shape) != (hq, T) or \
                not lse.is_contiguous():
            raise ValueError("lse must be a contiguous float32 [heads, tokens] tensor on the device of q")
        lp = lse.data_ptr()
    n = cu_seqlens.numel() - 1
    if n < 0:
        raise ValueError("cu_seqlens must hold n_seqs + 1 offsets")
    cu = _int32(cu_seqlens, dev, n + 1, "cu_seqlens")
    used = 0 if seq_used is None else _int32(seq_used, dev, n, "seq_used")
    return _VARLEN_PACK(*qv, *kv, *vv, *ov, lp, cu, used, T, n, hq, shape[1], d, 1 if causal else 0,
                        d ** -0.5 if scale is None else scale), dev


def attn_varlen_fwd(q, k, v, cu_seqlens, causal: bool = True, scale: Optional[float] = None, seq_used=None, out=None,
                    return_lse: bool = False, stream=None):
    """Attention within each sample of a pack (C entry point ``attn_varlen_fwd``).  q
    [T, Hq, d], k and v [T, Hkv, d]: bf16 CUDA views, any token and head strides (the
    slices of one fused QKV output), Hq a multiple of Hkv, d a multiple of 16 up to 128.
    ``seq_used`` (int32 [n]): only the first seq_used[s] rows of sample s are rows and keys.
    ``scale``: 1/sqrt(d) unless given.  Returns out [T, Hq, d] (a new tensor unless given;
    rows that see no key are 0), with ``return_lse`` (out, lse): lse float32 [Hq, T], the
    natural logarithm of each row's sum, which the backward takes."""
    _torch or _load_torch()
    if out is None:
        out = _empty(q.shape, _bf16, q.device, stream)
    lse = _empty((q.shape[1], q.shape[0]), _f32t, q.device, stream) if return_lse else None
    desc, dev = _varlen_desc(q, k, v, out, lse, cu_seqlens, causal, scale, seq_used)
    _launch(load_library().attn_varlen_fwd, "attn_varlen_fwd", dev, stream, desc)
    return (out, lse) if return_lse else out


def attn_varlen_bwd(dout, q, k, v, out, lse, cu_seqlens, causal: bool = True, scale: Optional[float] = None,
                    seq_used=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of ``attn_varlen_fwd`` for the output gradient ``dout`` (C entry
    point ``attn_varlen_bwd``), with the ``out`` and ``lse`` that it returned and its other
    arguments.  dq, dk and dv are written whole (new tensors unless given; rows of no sample
    get 0).  ``workspace``: a CUDA tensor of at least 8 * T * Hq bytes; allocated through
    torch unless given."""
    _torch or _load_torch()
    if lse is None:
        raise ValueError("the backward needs the forward's lse (return_lse=True)")
    if dout is None:
        raise ValueError("dout is required")
    desc, dev = _varlen_desc(q, k, v, out, lse, cu_seqlens, causal, scale, seq_used)
    grads, packed = [], []
    for name, t, like in (("dout", dout, q), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is None:
            t = _empty(like.shape, _bf16, q.device, stream)
        elif t.shape != like.shape or t.get_device() != dev:
            raise ValueError("%s must have shape %s on %s" % (name, tuple(like.shape), q.device))
        packed += _view(t, name)
        grads.append(t)
    lib = load_library()
    if workspace is None:
        need = lib.attn_varlen_bwd_workspace_bytes(q.shape[0], q.shape[1])
        workspace = _empty(max(need, 0), _torch.uint8, q.device, stream, returned=False)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the device of q")
    _launch(lib.attn_varlen_bwd, "attn_varlen_bwd", dev, stream, desc, _GRADS_PACK(*packed), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return tuple(grads[1:])


def attn_fault() -> bool:
    """Whether a bounded wait inside an attention kernel has run out on the current device
    since the library was loaded or this was last called: results since then are invalid.
    Synchronises the device."""
    st = load_library().attn_fault()
    if st < 0:
        _check("attn_fault", st)
    return st != 0


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
        @torch.autograd.function.once_differentiable       # the kernels have no second derivative
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
    those that the kernels cannot address (broadcast ones) are copied.  Differentiable once: a
    second derivative raises an error."""
    global _Attn
    if _Attn is None:
        _Attn = _attn_function()
    return _Attn.apply(_rows(q), _rows(k), _rows(v), cu_seqlens, bool(causal), scale, seq_used)
