"""Slopes that a model holds as a parameter (no GPU): refused where autograd would owe them a gradient,
taken where it records nothing."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from packed_varlen_rope_gb300 import _attention as A  # noqa: E402

CU = torch.tensor([0, 3], dtype=torch.int32)


@pytest.fixture
def seen(monkeypatch):
    """What the forward's kernel is called with; it stands in as q^2."""
    calls = []

    def fwd(q, k, v, *a, **kw):
        calls.append(kw.get("distance_slopes"))
        return q.detach() ** 2, torch.zeros(2, 3)

    monkeypatch.setattr(A, "attn_varlen_fwd", fwd)
    return calls


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_evaluated_without_gradients(seen, mode):
    q, k, v = (torch.randn(3, 2, 16, requires_grad=True) for _ in range(3))
    slopes = torch.nn.Parameter(torch.tensor([0.5, 0.25]))
    with mode():
        out = A.apply_attn(q, k, v, CU, distance_slopes=slopes)
    assert not out.requires_grad and len(seen) == 1 and seen[0] is not None and torch.equal(seen[0], slopes)


def test_refused_where_a_gradient_is_recorded(seen):
    q, k, v = (torch.randn(3, 2, 16) for _ in range(3))
    slopes = torch.nn.Parameter(torch.tensor([0.5, 0.25]))
    with pytest.raises(ValueError, match="constants"):
        A.apply_attn(q, k, v, CU, distance_slopes=slopes)
    with torch.no_grad(), torch.enable_grad(), pytest.raises(ValueError, match="constants"):
        A.apply_attn(q, k, v, CU, distance_slopes=slopes)
    assert not seen
    A.apply_attn(q, k, v, CU, distance_slopes=slopes.detach())
    assert len(seen) == 1
