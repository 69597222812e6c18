"""ctypes binding of the rotation by several position axes (``include/rope_axes.h``):
argument marshalling only, in the manner of ``_binding``."""
from __future__ import annotations

import ctypes
import struct

from . import _attention as A
from . import _binding as B

ROPE_MAX_AXES = 4
ROPE_AXES_INTERLEAVED, ROPE_AXES_OWN_FREQUENCIES, ROPE_AXES_IDS_INT64 = 0x1, 0x2, 0x4

_NO_SECTIONS = (0,) * ROPE_MAX_AXES

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class RopeAxesDesc(ctypes.Structure):
    """Mirror of ``rope_axes`` in include/rope_axes.h."""

    _fields_ = [("position_ids", _vp), ("position_stride", _i64), ("n_axes", _i32), ("flags", _i32),
                ("sections", _i32 * ROPE_MAX_AXES)]


# packed in one go, as the attention's descriptors: the structures above and RopeQKDesc
_AXES_PACK = struct.Struct("@Pqii4i").pack
_QK_PACK = struct.Struct("@" + 4 * "Pqq" + "PiiiiPqqddPiiPPii").pack


def _declare(lib):
    """Signatures of the entry points (called by ``load_library``); descriptors packed as bytes."""
    lib.rope_axes_apply.argtypes = [_vp, _vp, _vp]
    lib.rope_kv_append_axes.argtypes = [_vp, _vp, _vp]
    lib.rope_axes_apply.restype = lib.rope_kv_append_axes.restype = ctypes.c_int


def check_sections(sections, head_dim: int):
    """``sections`` as a tuple of 1 to 4 counts that share head_dim/2 frequencies among the axes."""
    counts = tuple(map(int, sections))
    if not 1 <= len(counts) <= ROPE_MAX_AXES or min(counts) < 1 or sum(counts) != head_dim // 2:
        raise ValueError("sections must be 1 to %d positive counts that add up to head_dim/2 = %d" %
                         (ROPE_MAX_AXES, head_dim // 2))
    return counts


def pack_axes(position_ids, sections, T: int, dev: int, interleaved: bool, own_frequencies: bool) -> bytes:
    """The packed ``rope_axes`` of a call over T tokens on CUDA device ``dev`` (the sections' sum is
    checked by the library)."""
    if position_ids is None or sections is None:
        raise ValueError("position_ids and sections go together")
    n = len(sections)
    if not 1 <= n <= ROPE_MAX_AXES:
        raise ValueError("give 1 to %d sections" % ROPE_MAX_AXES)
    st, dtype = position_ids.stride(), position_ids.dtype
    flags = 0 if dtype is A._i32t else ROPE_AXES_IDS_INT64
    if (flags != 0 and dtype is not A._torch.int64) or position_ids.get_device() != dev or position_ids.shape != (n, T) or (st[1] != 1 and T > 1):
        raise ValueError("position_ids must be an int32 or int64 [%d axes, %d tokens] tensor with contiguous rows on the "
                         "device of q" % (n, T))
    if interleaved:
        flags |= ROPE_AXES_INTERLEAVED
    if own_frequencies:
        flags |= ROPE_AXES_OWN_FREQUENCIES
    return _AXES_PACK(position_ids.data_ptr(), st[0] if n > 1 else T, n, flags, *sections, *_NO_SECTIONS[n:])


def rope_axes_apply(q, k, theta: float, sections, position_ids, backward: bool = False, q_out=None, k_out=None,
                    position_scale: float = 1.0, cos_sin_cache=None, stream=None, interleaved: bool = False,
                    own_frequencies: bool = False):
    """Rotation by several position axes, e.g. (time, height, width) of image and video tokens
    (C entry point ``rope_axes_apply``).

    q, k: bf16 CUDA views [T, Hq, d] and [T, Hkv, d] with any token/head strides.
    ``position_ids``: int32 or int64 [axes, T] with contiguous rows (one row expanded to all axes
    too), a position of every token on each axis; a token
    with one outside [0, 2^24) is left out (give pad rows -1).  ``sections``: how many of the
    d/2 frequencies turn by each axis, consecutive ones, or with ``interleaved`` taking turns.
    ``own_frequencies``: every axis has the whole range of frequencies (theta^(-i/section)),
    not its part of one.  Where a token's positions are equal the result has the bits of
    ``rope_qk_apply``.  ``backward``: the transpose rotation.  A ``cos_sin_cache`` serves all
    axes (not with ``own_frequencies``).  Returns (q, k) in place, else (q_out, k_out)."""
    A._torch or A._load_torch()
    qv, kv = A._view(q, "q"), A._view(k, "k")
    (T, hq, d), (Tk, hkv, dk), dev = q.shape, k.shape, q.get_device()
    if Tk != T or dk != d or k.get_device() != dev:
        raise ValueError("q and k must share tokens, head_dim and device")
    qo = ko = (0, 0, 0)
    if q_out is not None or k_out is not None:
        if q_out is None or k_out is None:
            raise ValueError("give both q_out and k_out, or neither (in place)")
        if q_out.shape != q.shape or k_out.shape != k.shape or q_out.get_device() != dev or k_out.get_device() != dev:
            raise ValueError("q_out/k_out must have the shapes and device of q/k")
        qo, ko = A._view(q_out, "q_out"), A._view(k_out, "k_out")
    axes = pack_axes(position_ids, check_sections(sections, d), T, dev, interleaved, own_frequencies)
    ref = None if cos_sin_cache is None else B._cache_arg(cos_sin_cache, d, q.device)
    desc = _QK_PACK(*qv, *kv, *qo, *ko, 0, 0, hq, hkv, d, 0, T, 0, theta, position_scale,
                    0 if ref is None else ctypes.addressof(ref.contents), 1 if backward else 0, 0, 0, 0, 0, 0)
    A._launch(B.load_library().rope_axes_apply, "rope_axes_apply", dev, stream, desc, axes)
    return (q, k) if q_out is None else (q_out, k_out)


_RopeAxes = None


def _axes_function():
    import torch

    class RopeAxes(torch.autograd.Function):
        """Autograd wrapper: forward rotates q and k in place (they are marked dirty); backward
        applies the transpose rotation to the incoming gradients."""

        @staticmethod
        def forward(ctx, q, k, position_ids, theta, sections, options):
            rope_axes_apply(q, k, theta, sections, position_ids, **options)
            ctx.mark_dirty(q, k)
            ctx.save_for_backward(position_ids)
            ctx.args = (theta, sections, options)
            return q, k

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dq, dk):
            (position_ids,) = ctx.saved_tensors
            theta, sections, options = ctx.args
            dq, dk = dq.contiguous(), dk.contiguous()      # e.g. broadcast (stride 0) gradients
            out = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (dq, dk)]
            # rows that the forward left out pass their gradient through: copied
            rope_axes_apply(dq, dk, theta, sections, position_ids, backward=True, q_out=out[0], k_out=out[1], **options)
            return out[0], out[1], None, None, None, None

    return RopeAxes


def apply_rope_axes(q, k, theta: float, sections, position_ids, cos_sin_cache=None, position_scale: float = 1.0,
                    interleaved: bool = False, own_frequencies: bool = False):
    """Differentiable in-place ``rope_axes_apply``, of tensors of their own: autograd refuses views
    (the slices of one projection's output) rotated in place together, clone them.  Differentiable
    once: a second derivative raises."""
    global _RopeAxes
    if _RopeAxes is None:
        _RopeAxes = _axes_function()
    options = dict(cos_sin_cache=cos_sin_cache, position_scale=float(position_scale), interleaved=bool(interleaved),
                   own_frequencies=bool(own_frequencies))
    return _RopeAxes.apply(q, k, position_ids, float(theta), tuple(int(x) for x in sections), options)
