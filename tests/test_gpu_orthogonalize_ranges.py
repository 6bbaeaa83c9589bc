"""The orthogonalisation at the ends of its range, against the steps in 64 bits; every test through both
libraries."""
import math

import pytest
import torch

import layer_ref as R
from nvfp4_testlib import need_gpu

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["release", "checked"], autouse=True)
def _library(request):
    need_gpu()
    if request.param == "release":
        yield
    else:
        with B.bounds_checked():
            yield


def test_zeros_with_any_eps():
    g = torch.randn(3, 50, 70, device="cuda")
    g[1] = 0
    for eps in (1e-300, 1e-100, 1e-60, 1e30):
        assert not B.orthogonalize(g, eps=eps)[1].any()
        assert not B.orthogonalize(g[1], eps=eps).any()


# The error of a value, as far as it goes back to the FP16 operands, is a sum over their roundings, of which
# R.orthogonalize_rounded draws one with all of them at half a step: s, its square's mean over 8 draws.  Up to 64 terms
# cannot pass 8 s^(1/2); more add up to a normal law of at most 0.58 of that.  A value among many like it is held to
# the mean of its row, column or matrix where the draws say less.  The result's rounding to bf16 adds 2^-8 of a value
# (and 2^-15 in second order, which covers the 22 bits of X and FP32).
#   Where ||G|| is far below eps little but that is left, and what counts are the values near zero.  X, at
# most t = ||G|| / (||G|| + eps), times a power of two that brings it to 1/2 .. 1, times S ~ n^(1/2), is held to 2^-36;
# A and B, to 2^-37 and 2^-35, act on a column of X, t n^(-1/2) large.  Every later step multiplies by |a| at most, or
# the singular values reach 1, and 5 steps add up to 12 * 2^-36 for X and, at 6 deviations of their sums over a
# column, 5 (3.5 + 4.8) 2^-35 for the others: under 128 * 2^-36 of t prod |a| n^(-1/2), S being within 2^(1/2) of n^(1/2).
def _check(out, g, eps, what, steps=5, coefficients=R.MUON):
    g3, o3 = (g, out) if g.dim() == 3 else (g[None], out[None])
    kw = dict(eps=eps, steps=steps, coefficients=coefficients)
    grown = math.prod(abs(c[0]) for c in ([coefficients] * steps if not hasattr(coefficients[0], "__len__")
                                          else coefficients))
    for e in range(g3.shape[0]):
        ref = R.orthogonalize(g3[e], **kw)
        s = sum((R.orthogonalize_rounded(g3[e], seed=i, **kw) - ref).square() for i in range(8)) / 8
        around = s.mean(1, keepdim=True).maximum(s.mean(0, keepdim=True)).clamp(min=float(s.mean()))
        norm = float(g3[e].double().norm())
        held = 128 * 2.0 ** -36 * norm / (norm + eps) * grown / max(ref.shape) ** 0.5
        bound = 2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs() + 8 * s.maximum(around).sqrt() + held + 2.0 ** -126
        off = (o3[e].double() - ref).abs()
        assert (off <= bound).all(), (what, e, float((off / bound).max()),
                                      float((o3[e].double() - ref).norm() / ref.norm()))


def _normal(shape, norm, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float64)
    return (g * (norm / g.square().sum((-2, -1), keepdim=True).sqrt())).float()


# (through narrow tiles, by clusters and alone, single CTAs, pairs; turned ones too)
@pytest.mark.parametrize("rows,cols,norms", [
    (1, 5, (1e-7, 1e-10, 1e-13, 1e-14, 1e-16, 1e-18, 1e-30)), (33, 17, (1e-7, 1e-13, 1e-16, 1e-18, 1e-30)),
    (256, 512, (1e-7, 1e-10, 1e-13, 1e-14, 1e-16, 1e-18, 1e-30)), (512, 256, (1e-10, 1e-14, 1e-18)),
    (640, 2047, (1e-10, 1e-16)), (2048, 640, (1e-10, 1e-16)), (2304, 2301, (1e-10, 1e-16))])
def test_gradients_far_below_eps(rows, cols, norms):
    for norm in norms:
        _check_one(rows, cols, norm)


def _check_one(rows, cols, norm):
    g = _normal((rows, cols), norm)
    _check(B.orthogonalize(g), g, 1e-7, (rows, cols, norm))


def test_a_small_matrix_in_a_batch_of_ordinary_ones():
    g = _normal((6, 200, 320), 1.0)
    want = B.orthogonalize(g)
    for i, norm in ((1, 1e-16), (4, 1e-11), (5, 3e-8)):
        g[i] *= norm
    out = B.orthogonalize(g)
    _check(out, g, 1e-7, "batch")
    for i in (0, 2, 3):
        assert torch.equal(out[i], want[i])


@pytest.mark.parametrize("eps", [0.5, 3.0, 1e3, 1e12, 1e30])
def test_eps_above_the_norm(eps):
    g = _normal((130, 260), 2.0)
    _check(B.orthogonalize(g, eps=eps), g, eps, eps)
    # a power of two on both changes nothing
    assert torch.equal(B.orthogonalize(g * 2.0 ** -40, eps=eps * 2.0 ** -40), B.orthogonalize(g, eps=eps))


def test_steps_that_bring_small_gradients_up():
    """From far below eps to where the singular values stay: X's own factor is 1 at the end."""
    g = _normal((96, 160), 1e-11)
    for steps in (1, 6, 9, 14):
        _check(B.orthogonalize(g, steps=steps), g, 1e-7, steps, steps=steps)
    mixed = [(4.0, -6.0, 2.5), (0.25, 0.0, 0.0), R.MUON, (0.0, 1.0, 0.0), (1.875, -1.25, 0.375)]
    _check(B.orthogonalize(g, coefficients=mixed), g, 1e-7, "mixed", coefficients=mixed)
