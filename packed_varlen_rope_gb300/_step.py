"""ctypes binding of a serving step's page tables (``include/paged_step.h``): argument
marshalling only, in the manner of ``_binding``."""
from __future__ import annotations

import ctypes

from . import _binding as B

PAGED_EXPORTS = ("paged_kv_step",)

STEP_NO_PAGES, STEP_TABLE_FULL, STEP_STACK_FULL, STEP_TOKENS_PAST_END, STEP_NEGATIVE_LENGTH = 0x1, 0x2, 0x4, 0x8, 0x10

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class PagedKVStepDesc(ctypes.Structure):
    """Mirror of ``paged_kv_step_desc`` in include/paged_step.h."""

    _fields_ = [("free_pages", _vp), ("free_count", _vp), ("count_out", _vp), ("page_table", _vp),
                ("page_table_stride", _i64), ("past_lens", _vp), ("new_lens", _vp), ("finished", _vp),
                ("cu_seqlens", _vp), ("kv_lens", _vp), ("slots", _vp), ("status", _vp), ("n_free_max", _i64),
                ("max_tokens", _i64), ("n_seqs", _i32), ("max_pages", _i32), ("page_size", _i32), ("reserved", _i32)]


def _declare(lib):
    """Signature of the entry point (called by ``load_library``)."""
    lib.paged_kv_step.argtypes = [ctypes.POINTER(PagedKVStepDesc), _vp]
    lib.paged_kv_step.restype = ctypes.c_int


def paged_kv_step(free_pages, free_count, page_table, past_lens, new_lens, page_size: int, max_tokens: int = 0,
                  finished=None, count_out=None, cu_seqlens=None, kv_lens=None, slots=None, status=None, stream=None):
    """The bookkeeping of one serving step over a paged cache, on the device (C entry point
    ``paged_kv_step``): finished sequences give their pages back, the growing ones get theirs.

    ``free_pages`` (int32 [capacity]) is a stack of free page ids with ``free_count`` (int32 [1])
    in use; ``page_table`` (int32 [n, max_pages]) is updated in place; ``past_lens`` and
    ``new_lens`` (int32 [n]) count each row's tokens in the cache and those this step adds.
    ``finished`` (int32 [n], nonzero: over): the row's pages go onto the stack first, and the row
    starts empty.  All on the device.  Returns (cu_seqlens [n + 1], kv_lens [n], slots): what
    ``rope_kv_append`` and ``attn_paged`` take, and the place page * page_size + offset of each of
    ``max_tokens`` new tokens (int64, -1 where there is none; None for max_tokens 0).
    ``count_out``: the count after the step (``free_count`` itself unless given).  ``status``
    (int32 [1]) receives STEP_* bits: no pages left, a row longer than the table, a stack or the
    slots too small, a negative length."""
    import torch

    dev, n = page_table.device, past_lens.numel()
    if dev.type != "cuda" or page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != n or \
            (page_table.shape[1] > 1 and page_table.stride(1) != 1) or (n > 1 and page_table.stride(0) < 0):
        raise ValueError("page_table must be a CUDA int32 [n_seqs, max_pages] tensor with contiguous rows")
    max_tokens = int(max_tokens)
    if slots is not None:
        max_tokens = slots.numel()
    elif max_tokens > 0:
        slots = B._empty(max_tokens, torch.int64, dev, stream)
    if cu_seqlens is None:
        cu_seqlens = B._empty(n + 1, torch.int32, dev, stream)
    if kv_lens is None:
        kv_lens = B._empty(n, torch.int32, dev, stream)
    if count_out is None:
        count_out = free_count
    for name, t, size, dtype in (("free_pages", free_pages, free_pages.numel(), torch.int32),
                                 ("free_count", free_count, 1, torch.int32), ("count_out", count_out, 1, torch.int32),
                                 ("past_lens", past_lens, n, torch.int32), ("new_lens", new_lens, n, torch.int32),
                                 ("finished", finished, n, torch.int32), ("cu_seqlens", cu_seqlens, n + 1, torch.int32),
                                 ("kv_lens", kv_lens, n, torch.int32), ("slots", slots, max_tokens, torch.int64),
                                 ("status", status, 1, torch.int32)):
        if t is not None and (t.dtype != dtype or t.device != dev or t.numel() != size or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous %s tensor of %d values on %s" % (name, dtype, size, dev))
    desc = PagedKVStepDesc(B._ptr(free_pages), B._ptr(free_count), B._ptr(count_out), B._ptr(page_table),
                           page_table.stride(0), B._ptr(past_lens), B._ptr(new_lens), B._ptr(finished), B._ptr(cu_seqlens),
                           B._ptr(kv_lens), B._ptr(slots), B._ptr(status), free_pages.numel(), max_tokens, n,
                           page_table.shape[1], int(page_size), 0)
    st = B._on(dev, B.load_library().paged_kv_step, ctypes.byref(desc), B._stream(stream, dev))
    B._check("paged_kv_step", st)
    return cu_seqlens, kv_lens, slots
