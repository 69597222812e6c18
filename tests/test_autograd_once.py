"""Derivatives of derivatives (no GPU): the backward passes are kernels outside autograd, so a second
derivative through them must raise, not come out with their terms missing."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import packed_varlen_rope_gb300 as pr  # noqa: E402
from packed_varlen_rope_gb300 import _attention as A  # noqa: E402


def assert_second_derivative_raises(out, x):
    """``out`` is a function of x; the first derivative comes out, a second one raises, also
    where other terms of the loss have one."""
    (g,) = torch.autograd.grad(out.square().sum(), x, create_graph=True)
    assert g.shape == x.shape
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (g.square().sum() + x.square().sum()).backward()


def test_attention(monkeypatch):
    """The kernels stand in as o = q^2 and its gradient, detached as theirs are."""
    monkeypatch.setattr(A, "attn_varlen_fwd", lambda q, k, v, *a, **kw: (q.detach() ** 2, torch.zeros(2, 3)))
    monkeypatch.setattr(A, "attn_varlen_bwd", lambda do, q, k, v, *a, **kw:
                        ((2 * q * do).detach(), torch.zeros_like(k), torch.zeros_like(v)))
    q, k, v = (torch.randn(3, 2, 16, requires_grad=True) for _ in range(3))
    out = A._attn_function().apply(q, k, v, torch.tensor([0, 3], dtype=torch.int32), True, None, None)
    assert_second_derivative_raises(out, q)
