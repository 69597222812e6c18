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


def test_rotation(monkeypatch):
    """The kernel stands in as a product by 2, in place or into q_out and k_out."""
    def double(q, k, theta, q_out=None, k_out=None, **kw):
        (q if q_out is None else q_out).data.copy_(2 * q.detach())
        (k if k_out is None else k_out).data.copy_(2 * k.detach())

    monkeypatch.setattr(pr, "rope_qk_apply", double)
    q, k = torch.randn(3, 2, 16, requires_grad=True), torch.randn(3, 1, 16)
    out, _ = pr._autograd_function().apply(q.clone(), k, 1e4, torch.tensor([0, 3], dtype=torch.int32), None, 0, 1.0, None,
                                           None, None)
    assert_second_derivative_raises(out, q)


def test_glu(monkeypatch):
    """The kernels stand in as e^2 g and its gradient."""
    monkeypatch.setattr(pr, "glu_fwd", lambda kind, e, g: e.detach() ** 2 * g.detach())
    monkeypatch.setattr(pr, "glu_bwd", lambda kind, dh, e, g: ((2 * e * g * dh).detach(), (e ** 2 * dh).detach()))
    e, g = torch.randn(3, 8, requires_grad=True), torch.randn(3, 8)
    assert_second_derivative_raises(pr._glu_function().apply("swiglu", e, g), e)
