"""ctypes binding of a serving step's page tables (``include/paged_step.h``): argument
marshalling only, in the manner of ``_binding``."""
from __future__ import annotations

import ctypes
import struct

from . import _attention as A
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


_STEP_PACK = struct.Struct("@PPPPqPPPPPPPqqiiii").pack


def _declare(lib):
    """Signature of the entry point (called by ``load_library``); the descriptor packed as bytes."""
    lib.paged_kv_step.argtypes = [_vp, _vp]
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
    torch = A._torch or A._load_torch()
    i32 = A._i32t
    st, shape, dev = page_table.stride(), page_table.shape, page_table.get_device()
    n = past_lens.numel()
    if dev < 0 or page_table.dtype is not i32 or len(shape) != 2 or shape[0] != n or (shape[1] > 1 and st[1] != 1) or \
            (n > 1 and st[0] < 0):
        raise ValueError("page_table must be a CUDA int32 [n_seqs, max_pages] tensor with contiguous rows")
    device, max_tokens = page_table.device, int(max_tokens)
    if slots is not None:
        max_tokens = slots.numel()
        if slots.dtype is not torch.int64 or slots.get_device() != dev or not slots.is_contiguous():
            raise ValueError("slots must be a contiguous int64 tensor on %s" % device)
    elif max_tokens > 0:
        slots = _new(torch, max_tokens, torch.int64, device, stream)
    if cu_seqlens is None:
        cu_seqlens = _new(torch, n + 1, i32, device, stream)
        cu = cu_seqlens.data_ptr()
    else:
        cu = _ints(cu_seqlens, dev, n + 1, "cu_seqlens")
    if kv_lens is None:
        kv_lens = _new(torch, n, i32, device, stream)
        kv = kv_lens.data_ptr()
    else:
        kv = _ints(kv_lens, dev, n, "kv_lens")
    capacity = free_pages.numel()
    count = _ints(free_count, dev, 1, "free_count")
    desc = _STEP_PACK(_ints(free_pages, dev, capacity, "free_pages"), count,
                      count if count_out is None else _ints(count_out, dev, 1, "count_out"), page_table.data_ptr(), st[0],
                      _ints(past_lens, dev, n, "past_lens"), _ints(new_lens, dev, n, "new_lens"),
                      0 if finished is None else _ints(finished, dev, n, "finished"),
                      cu, kv, 0 if slots is None else slots.data_ptr(),
                      0 if status is None else _ints(status, dev, 1, "status"), capacity, max_tokens, n, shape[1], int(page_size), 0)
    A._launch(B.load_library().paged_kv_step, "paged_kv_step", dev, stream, desc)
    return cu_seqlens, kv_lens, slots


def _new(torch, n: int, dtype, device, stream):
    return torch.empty(n, dtype=dtype, device=device) if stream is None else B._empty(n, dtype, device, stream)


def _ints(t, dev: int, n: int, what: str) -> int:
    """Pointer of a contiguous int32 tensor of n values on CUDA device ``dev``."""
    if t.dtype is not A._i32t or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of %d values on the device of page_table" % (what, n))
    return t.data_ptr()
