"""Rules on attention scores without a GPU: the tests' formulas against differences, the constants of
the tanh, the binding's structure, refusals before any launch, the autograd wrapper."""
from __future__ import annotations

import ctypes
import os
import re
import struct
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from rule_util import sample_reference, scores, visible  # noqa: E402
from test_attn_abi_host import ERR_ALIGN, ERR_NULL, ERR_THETA, ERR_UNSUPPORTED, OK, grads, paged, varlen  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "packed_varlen_rope_gb300", "csrc")
BASE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from packed_varlen_rope_gb300 import build, load_library

    build.build()
    return load_library()


def plain(q, k, v, scale, cap, slopes, prefix, causal):
    """The definition, differentiable: [n, H, d] of H query heads to as many outputs."""
    g = q.shape[1] // k.shape[1]
    Q, K, V = (x.transpose(0, 1) for x in (q, k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)))
    s, _ = scores(Q, K, scale, cap, slopes, torch.arange(q.shape[0]))
    s = s.masked_fill(~visible(q.shape[0], k.shape[0], causal, prefix, q.device), float("-inf"))
    return (s.softmax(-1) @ V).transpose(0, 1)


@pytest.mark.parametrize("cap,sloped,prefix,causal", [(3.0, False, None, True), (0.0, True, None, False),
                                                      (0.0, False, 4, True), (2.0, True, 5, True)])
def test_formulas_against_differences(cap, sloped, prefix, causal):
    """Gradients that the reference writes out, against autograd's and against central differences."""
    gen = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(9, h, 16, generator=gen, dtype=torch.float64) for h in (4, 2, 2, 4))
    slopes = torch.tensor([0.5, 0.25, 1.0, 0.03], dtype=torch.float64) if sloped else None
    f = lambda a, b, c: (plain(a, b, c, 0.7, cap, slopes, prefix, causal) * do).sum()       # noqa: E731
    ref = sample_reference(q, k, v, 0.7, cap, slopes, prefix, causal, do)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    f(*leaves).backward()
    for x, name in zip(leaves, ("dq", "dk", "dv")):
        assert float((x.grad - ref[name][0]).abs().max()) < 1e-12
    for i, name in enumerate(("dq", "dk", "dv")):
        way = torch.randn((q, k, v)[i].shape, generator=gen, dtype=torch.float64)
        eps = 1e-5
        args = [[x + (sign * eps * way if j == i else 0) for j, x in enumerate((q, k, v))] for sign in (1, -1)]
        slope = (f(*args[0]) - f(*args[1])) / (2 * eps)
        assert abs(float(slope - (ref[name][0] * way).sum())) < 1e-7


def kernel_constants(name, n):
    text = open(os.path.join(CSRC, "score_rule.cuh")).read()
    return np.array([float(re.search(r"%s%d = ([-0-9.e]+)f" % (name, i), text).group(1)) for i in range(n)])


@pytest.fixture(scope="module")
def fit_tanh():
    sys.path.insert(0, CSRC)
    try:
        import fit_tanh as module
    finally:
        sys.path.remove(CSRC)
    return module


def test_tanh_constants_are_the_fits(fit_tanh):
    for name, want in (("kNear", fit_tanh.near()), ("kSmall", fit_tanh.small()), ("kTanh", fit_tanh.large())):
        got = kernel_constants(name, len(want))
        assert np.all(np.abs(got - want) <= 1e-9 * np.abs(want) + 1e-10)
    assert fit_tanh.near_error(fit_tanh.small(), end=fit_tanh.SMALL) < 5.6e-6
    assert fit_tanh.near_error(fit_tanh.near()) < 6.7e-6 and fit_tanh.large_error(fit_tanh.large()) < 6.1e-7


@pytest.mark.parametrize("cap,scale", [(50.0, 0.088), (128.0, 0.125), (1.0, 1.0), (0.03, 20.0)])
@pytest.mark.parametrize("name,end", [("kNear", 0.8), ("kSmall", 0.5)])
def test_near_forms_in_binary32(fit_tanh, cap, scale, name, end):
    """Step by step: within 7e-6 of the cap up to 0.8 or half of it, and the factor within 2e-5."""
    f = np.float32
    a, k = f(scale) / f(cap), f(cap) * f(1.4426950408889634)
    assert end == {"kNear": fit_tanh.NEAR, "kSmall": fit_tanh.SMALL}[name]
    coef = [f(float(k) * float(a) ** (2 * i + 1) * x) for i, x in enumerate(kernel_constants(name, 4 if name == "kNear" else 3))]
    s = np.linspace(-end, end, 200001).astype(f) * (f(1) / a)
    z = s * s
    p = np.full_like(z, coef[-1])
    for x in coef[-2::-1]:
        p = z * p + x
    x = s * p
    t = np.tanh(s.astype(np.float64) * scale / cap)
    assert np.max(np.abs(x.astype(np.float64) / 1.4426950408889634 - cap * t)) < 7e-6 * cap
    unit = k * k
    factor = x * x - unit
    assert np.max(np.abs(-factor.astype(np.float64) / float(unit) - (1 - t * t))) < 2e-5


def test_other_forms_in_binary32():
    """Step by step: the form of every score within a few units of 2^-23 of the cap, that of large
    caps below 7e-7 of the score; their factors."""
    f = np.float32
    u = np.concatenate([-np.linspace(1e-3, 20, 100001), np.linspace(1e-3, 20, 100001)]).astype(f)
    exact = np.tanh(u.astype(np.float64))
    q = f(1) / (f(1) + np.exp2(f(2 * 1.4426950408889634) * u))
    assert np.max(np.abs(f(1) - f(2) * q - exact)) < 4 * 2.0 ** -23
    factor = -(q * (q * f(4) - f(4))).astype(np.float64)
    one_less = 1 / np.cosh(u.astype(np.float64)) ** 2
    # 1 - q cancels where q is near 1: absolute there
    assert np.max(np.abs(factor - one_less) / (one_less + 2.0 ** -6)) < 2.0 ** -15
    c = kernel_constants("kTanh", 6).astype(f)
    u = np.linspace(1e-6, 1, 200001).astype(f)
    z = u * u
    p = np.full_like(z, c[5])
    for i in (4, 3, 2, 1, 0):
        p = z * p + c[i]
    t = u * p
    exact = np.tanh(u.astype(np.float64))
    assert np.max(np.abs(t / exact - 1)) < 9e-7
    assert np.max(np.abs((f(1) - t * t) - (1 - exact ** 2))) < 2.0 ** -19


def test_structure_matches(tmp_path):
    from packed_varlen_rope_gb300 import AttnScoreRule, _attention as A

    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "attn.h"\nint main(void) {\n'
                   'printf("%zu", sizeof(attn_score_rule));\n' +
                   "".join('printf(" %%zu", offsetof(attn_score_rule, %s));\n' % f[0] for f in AttnScoreRule._fields_) +
                   "return 0; }\n")
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                           str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [ctypes.sizeof(AttnScoreRule)] + [getattr(AttnScoreRule, f[0]).offset for f in AttnScoreRule._fields_]
    assert A._RULE_PACK.__self__.size == ctypes.sizeof(AttnScoreRule)
    r = AttnScoreRule.from_buffer_copy(A._RULE_PACK(1, 2, 0.5, 0))
    assert (r.slopes, r.prefix, r.cap, r.reserved) == (1, 2, 0.5, 0)
    assert struct.calcsize("@PPfi") == 24


@pytest.mark.parametrize("kw,desc,want", [
    (dict(cap=-1.0), {}, ERR_THETA), (dict(cap=float("nan")), {}, ERR_THETA), (dict(cap=float("inf")), {}, ERR_THETA),
    (dict(cap=3e38), {}, ERR_THETA), (dict(cap=1e-39), {}, ERR_THETA), (dict(cap=1e30), dict(scale=1e-12), ERR_THETA),
    (dict(cap=1e-20), dict(scale=1e20), ERR_THETA), (dict(reserved=1), {}, ERR_UNSUPPORTED),
    (dict(slopes=BASE + 2), {}, ERR_ALIGN), (dict(prefix=BASE + 1), {}, ERR_ALIGN),
    (dict(prefix=BASE), dict(causal=0), ERR_UNSUPPORTED),
])
def test_rule_refusals(lib, kw, desc, want):
    from packed_varlen_rope_gb300 import AttnScoreRule

    rule = AttnScoreRule(**kw)
    ref, a = ctypes.byref, varlen(**desc)
    assert lib.attn_varlen_fwd_rule(ref(a), ref(rule), None) == want
    assert lib.attn_varlen_bwd_rule(ref(a), ref(grads()), ref(rule), BASE + (1 << 38), 1 << 20, None) == want
    assert lib.attn_paged_rule(ref(paged(**desc)), ref(rule), BASE + (1 << 38), 1 << 40, None) == want


def test_nothing_to_do(lib):
    from packed_varlen_rope_gb300 import AttnScoreRule

    rule, ref = AttnScoreRule(cap=30.0), ctypes.byref
    assert lib.attn_varlen_fwd_rule(ref(varlen(total_tokens=0)), ref(rule), None) == OK
    assert lib.attn_paged_rule(ref(paged(total_tokens=0)), ref(rule), None, 0, None) == OK
    assert lib.attn_varlen_fwd_rule(None, ref(rule), None) == ERR_NULL
    assert lib.attn_varlen_bwd_rule(ref(varlen()), None, ref(rule), None, 0, None) == ERR_NULL
    assert lib.attn_paged_rule(None, ref(rule), None, 0, None) == ERR_NULL


def test_second_derivative_raises_and_the_rule_reaches_the_backward(monkeypatch):
    from packed_varlen_rope_gb300 import _attention as A

    seen = {}
    monkeypatch.setattr(A, "attn_varlen_fwd", lambda q, k, v, *a, **kw: (q.detach() ** 2, torch.zeros(2, 3)))

    def bwd(do, q, k, v, *a, **kw):
        seen.update(kw)
        return (2 * q * do).detach(), torch.zeros_like(k), torch.zeros_like(v)

    monkeypatch.setattr(A, "attn_varlen_bwd", bwd)
    q, k, v = (torch.randn(3, 2, 16, requires_grad=True) for _ in range(3))
    slopes, prefix = torch.tensor([0.5, 0.25]), torch.tensor([2], dtype=torch.int32)
    out = A._attn_function().apply(q, k, v, torch.tensor([0, 3], dtype=torch.int32), True, None, None, 30.0, slopes, prefix)
    (g,) = torch.autograd.grad(out.square().sum(), q, create_graph=True)
    assert seen["score_cap"] == 30.0 and torch.equal(seen["distance_slopes"], slopes) and torch.equal(seen["prefix_lens"], prefix)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.square().sum().backward()
    with pytest.raises(ValueError):
        A.apply_attn(q, k, v, torch.tensor([0, 3], dtype=torch.int32), distance_slopes=slopes.requires_grad_())


@pytest.mark.parametrize("cap", [1e-50, -1e-50, 1e-40])
def test_a_cap_that_would_be_packed_as_none(cap):
    from packed_varlen_rope_gb300 import _attention as A

    with pytest.raises(ValueError, match="score_cap"):
        A._rule(cap, None, None, None, 0, 1)


def test_every_rule_has_an_instance():
    """The rules that the build compiles are those that the dispatch names."""
    from packed_varlen_rope_gb300 import build

    text = open(os.path.join(CSRC, "attn_internal.h")).read()
    declared = sorted(int(x) for x in re.findall(r"^PVR_DECLARE_RULE\((\d)\)", text, flags=re.M))
    assert all(sorted(rules) == declared for rules in build.RULES.values())
    assert sorted(int(x) for x in re.findall(r"integral_constant<int, (\d)>\{\}", text)) == declared
