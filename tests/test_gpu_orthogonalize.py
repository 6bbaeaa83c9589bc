"""GPU parity of the Newton-Schulz orthogonalisation against the steps in 64 bits; every test through
both libraries."""
import os
import subprocess
import sys

import pytest
import torch

import layer_ref as R
from nvfp4_testlib import need_gpu

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(params=["release", "checked"], autouse=True)
def _library(request):
    need_gpu()
    if request.param == "release":
        yield
    else:
        with B.bounds_checked():
            yield


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# To first order a value of the result is off by sum_k c_k d_k over the roundings d_k of the products'
# operands, |d_k| at most half a step of FP16 (the FP32 accumulators and state add 2^-13 of that each).
# R.orthogonalize_rounded gives that sum for d_k = half a step with a random sign: its rms over draws is
# s = (sum c_k^2)^(1/2) half a step, which 8 draws estimate.  The error is at most sum |c_k| half a step, which
# N terms of any size make N^(1/2) s: up to 64 terms cannot pass 8 s.  With more the real roundings, spread
# over the interval (rms 3^(-1/2) of its end), add up to a normal law of deviation 0.58 s, of which 8 s is 14.
# A value among many like it is held to the rms of its row, column or matrix where the draws say less.  The
# norm of the whole error is a sum over all values: 0.58 of that of s, or s itself where few values count; 1.2
# covers second orders.  The result's own rounding to bf16 adds half a step, 2^-8, of each value.
def _check(out, g, what="", **kw):
    g3 = g if g.dim() == 3 else g[None]
    o3 = out if out.dim() == 3 else out[None]
    assert out.dtype == torch.bfloat16 and out.shape == g.shape
    for e in range(g3.shape[0]):
        ref = R.orthogonalize(g3[e], **kw)
        s = sum((R.orthogonalize_rounded(g3[e], seed=i, **kw) - ref).square() for i in range(8)) / 8
        err = ((o3[e].double() - ref).abs() - 2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs()).clamp(min=0)
        floor = 2.0 ** -126
        assert err.norm() <= 1.2 * s.sum().sqrt() + floor, (what, e, float(err.norm() / s.sum().sqrt()))
        around = s.mean(1, keepdim=True).maximum(s.mean(0, keepdim=True)).clamp(min=float(s.mean()))
        bound = 8 * s.maximum(around).sqrt() + floor
        bad = ~(err <= bound)
        assert not bad.any(), (what, e, int(bad.sum()), float((err / bound).max()))


def _gradient(shape, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 1e-3 * torch.randn(shape, generator=g, device="cuda")
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.005, 30 * x, x).to(dtype)


SIZES = [(1, 1), (1, 7), (9, 1), (16, 16), (64, 64), (127, 129), (128, 128), (129, 127), (130, 260), (257, 255),
         (300, 1000), (1000, 333), (512, 512), (64, 4096), (4097, 65), (640, 2048)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_against_64_bits(rows, cols, dtype):
    g = _gradient((rows, cols), dtype, rows + cols)
    st = _status()
    _check(B.orthogonalize(g, dev_status=st), g, (rows, cols))
    assert int(st) == 0


@pytest.mark.parametrize("rows,cols", [(2500, 2300), (2304, 4608), (5000, 1900), (2303, 2616), (3100, 2312),
                                       (2300, 2601)])
def test_sizes_that_take_pairs(rows, cols):
    g = _gradient((rows, cols), seed=1)
    _check(B.orthogonalize(g), g, (rows, cols))


@pytest.mark.parametrize("batch,rows,cols", [(3, 40, 100), (5, 200, 130), (2, 1, 1), (17, 384, 256), (1, 70, 70),
                                             (12, 520, 1300), (200, 16, 24)])
def test_batches(batch, rows, cols):
    g = _gradient((batch, rows, cols), seed=batch)
    g[batch // 2] *= 1e4  # each has a norm of its own
    _check(B.orthogonalize(g), g, (batch, rows, cols))


@pytest.mark.parametrize("kind", ["low rank", "rows", "columns", "one row", "orthogonal", "rank one", "few nonzero"])
@pytest.mark.parametrize("rows,cols", [(320, 512), (512, 320)])
def test_gradients_of_other_kinds(kind, rows, cols):
    torch.manual_seed(0)
    g = torch.randn(rows, cols, device="cuda")
    if kind == "low rank":
        g = torch.randn(rows, 8, device="cuda") @ torch.randn(8, cols, device="cuda") + 1e-2 * g
    elif kind == "rows":
        g = g * torch.logspace(-2, 0, rows, device="cuda")[:, None]
    elif kind == "columns":
        g = g * torch.logspace(-2, 0, cols, device="cuda")
    elif kind == "one row":
        g[1:] = 0
    elif kind == "orthogonal":
        g = torch.linalg.qr(g if rows >= cols else g.T)[0]
        g = (g if rows >= cols else g.T).contiguous()
    elif kind == "rank one":
        g = torch.randn(rows, 1, device="cuda") @ torch.randn(1, cols, device="cuda")
    else:
        g = g * (torch.rand(rows, cols, device="cuda") < 0.01)
    _check(B.orthogonalize(g), g, kind)


def test_steps_and_coefficients():
    g = _gradient((200, 300))
    for steps in (1, 2, 7):
        _check(B.orthogonalize(g, steps=steps), g, steps, steps=steps)
    taylor = (1.875, -1.25, 0.375)  # keeps 1 where it is
    _check(B.orthogonalize(g, steps=8, coefficients=taylor), g, "taylor", steps=8, coefficients=taylor)
    mixed = [(4.0, -6.0, 2.5), (3.4445, -4.7750, 2.0315), taylor]
    _check(B.orthogonalize(g, steps=3, coefficients=mixed), g, "mixed", steps=3, coefficients=mixed)
    _check(B.orthogonalize(g, eps=0.5), g, "eps", eps=0.5)
    # what it is for: singular values near 1
    s = torch.linalg.svdvals(B.orthogonalize(_gradient((256, 1024))).double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e30])
def test_gradients_of_any_size(scale):
    g = torch.randn(100, 90, device="cuda") * scale
    kw = dict(eps=0.0)
    _check(B.orthogonalize(g, **kw), g, scale, **kw)


def test_zeros_and_values_that_are_not_finite():
    g = _gradient((5, 60, 200))
    g[1] = 0
    clean = B.orthogonalize(g)
    assert not clean[1].any()
    g[3, 17, 5], g[4, 0, 0] = float("nan"), float("-inf")
    st = _status()
    out = B.orthogonalize(g, dev_status=st)
    assert int(st) == B.DEVSTAT_NONFINITE
    assert torch.equal(out[:3], clean[:3]) and not out[3:].any()
    for eps in (0.0, 1e-7):
        assert not B.orthogonalize(torch.zeros(33, 20, device="cuda"), eps=eps).any()


@pytest.mark.parametrize("rows,cols", [(96, 160), (160, 96), (75, 131), (131, 75), (75, 136), (139, 72), (900, 1000),
                                       (1200, 1001), (1201, 1000)])
def test_strides_and_what_lies_around(rows, cols):
    base = _gradient((3, rows, cols))
    want = B.orthogonalize(base)
    wide = torch.full((3, rows + 1, cols + 5), float("nan"), device="cuda")
    g = wide[:, :rows, 3:3 + cols]
    g.copy_(base)
    for pad, first in ((8, 0), (8, 8), (5, 0), (5, 3), (16, 1)):
        buf = torch.full((3, rows + 2, cols + 16 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:, 1:-1, first:first + cols]
        assert B.orthogonalize(g, out=out) is out
        assert torch.equal(out, want), (pad, first)
        out.fill_(7.0)
        assert (buf == 7.0).all(), (pad, first)
    # a matrix for all of a batch, and a row for all of a matrix
    one = base[:1].expand(3, rows, cols)
    assert torch.equal(B.orthogonalize(one), want[:1].expand(3, rows, cols))
    row = base[0, :1].expand(rows, cols)
    _check(B.orthogonalize(row), row.contiguous(), "row")
    # in place
    h = base.bfloat16()
    want = B.orthogonalize(h)
    B.orthogonalize(h, out=h)
    assert torch.equal(h, want)


def test_single_rows_and_matrices_of_any_stride():
    wide = _gradient((4, 6, 33))
    want = B.orthogonalize(wide[1:2, 2:3].contiguous())
    assert torch.equal(B.orthogonalize(wide[1:2, 2:3]), want)
    assert torch.equal(B.orthogonalize(wide[1, 2:3]), want[0])
    out = torch.zeros(4, 6, 33, dtype=torch.bfloat16, device="cuda")
    B.orthogonalize(wide[1:2, 2:3], out=out[3:4, 5:6])
    assert torch.equal(out[3:4, 5:6], want)
    out[3, 5] = 0
    assert not out.any()


def test_workspace_is_enough_and_no_state_is_kept():
    need = B.lib().nvfp4_orthogonalize_workspace_bytes(2, 200, 500)
    room = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    g = _gradient((2, 200, 500))
    want = B.orthogonalize(g)
    for fill in (0xFF, 0, 0x7C):
        room.fill_(fill)
        for first in (256, 16, 144):  # 16-byte aligned is enough
            assert torch.equal(B.orthogonalize(g, workspace=room[first:first + need]), want)
            assert (room[:first] == fill).all() and (room[first + need:] == fill).all()
            room.fill_(fill)


def test_on_another_stream_captured_and_replayed():
    g = _gradient((2, 300, 140))
    want = B.orthogonalize(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = B.orthogonalize(g, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    coefficients = [list(R.MUON) for _ in range(5)]
    with torch.cuda.graph(graph):
        captured = B.orthogonalize(g, coefficients=coefficients)
    coefficients[0][0] = 0.0  # read when the call was made
    for seed in range(3):
        g.copy_(_gradient((2, 300, 140), seed=seed + 5))
        want = B.orthogonalize(g)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, want)
    del graph


def test_two_calls_at_once():
    a, b = _gradient((700, 900), seed=1), _gradient((1500, 400), seed=2)
    want = B.orthogonalize(a), B.orthogonalize(b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        got = B.orthogonalize(a, stream=streams[0]), B.orthogonalize(b, stream=streams[1])
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_first_call_of_a_process_may_be_captured():
    code = """
import torch
from nvfp4_bit_quantized_03_b200 import binding as B
for shape in ((300, 200), (2304, 2304)):
    g = torch.randn(shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = B.orthogonalize(g)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, B.orthogonalize(g))
    del graph
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=300)


def test_gradients_with_an_exact_answer():
    """A permutation times a power of two: every step maps its singular values to one number."""
    n = 256
    g = torch.zeros(n, n, device="cuda")
    g[torch.arange(n), torch.randperm(n, device="cuda")] = 0.25
    s = 1 / n ** 0.5
    for a, b, c in [R.MUON] * 5:
        s = a * s + b * s ** 3 + c * s ** 5
    out = B.orthogonalize(g, eps=0.0)
    assert torch.equal(out != 0, g != 0)
    # A and B are diagonal, so all that moves a value is in 32 bits or X's 22.  2^-22 at each factor of the
    # terms b s^3 and c s^5, carried on by each step's slope s p'(s) / p(s), adds up to 69 * 2^-22 < 2^-12
    # over the five steps.  The answer is rounded to bf16: half a step is 2^-8.
    assert ((out[g != 0].double() - s).abs() <= (2.0 ** -8 + 2.0 ** -12) * s).all()
