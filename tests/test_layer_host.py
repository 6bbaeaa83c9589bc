"""Host-side checks of the operators around a layer's products that need no GPU: the references against
differences, sizes, and refusals before any work is queued (C ABI and binding)."""
import ctypes
import os
import re

import pytest
import torch

import layer_ref as R

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding

P = ctypes.c_void_p(0x10000)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_gradient_against_differences(interleaved):
    torch.manual_seed(0)
    T, H, D, eps = 3, 2, 32, 1e-3
    x, d = torch.randn(T, H, D).double(), torch.randn(T, H, D).double()
    w = torch.randn(D).double()
    table = R.rope_table(50, 16)
    p = torch.tensor([7, -1, 49], dtype=torch.int32)

    def loss(x, w):
        return (R.qk(x, w, eps, p, table, interleaved)[0] * d).sum()
    dx, dw, _ = R.qk_backward(d, x, w, eps, p, table, interleaved)
    h = 1e-5
    for _ in range(40):
        i = tuple(int(torch.randint(0, n, ())) for n in x.shape)
        e = torch.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for j in range(D):
        e = torch.zeros_like(w)
        e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-7
    # and against the other form of the rotation: complex products
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    n = 8
    row = table.double()[p.clamp(min=0).long()]
    phase = torch.complex(row[:, :n], row[:, n:])[:, None]
    a, b = (y[..., 0:16:2], y[..., 1:16:2]) if interleaved else (y[..., :n], y[..., n:16])
    z = torch.complex(a.contiguous(), b.contiguous()) * phase
    got = R.qk(x, w, eps, p, table, interleaved)[0]
    ga, gb = (got[..., 0:16:2], got[..., 1:16:2]) if interleaved else (got[..., :n], got[..., n:16])
    on = (p >= 0)
    assert torch.allclose(ga[on], z.real[on]) and torch.allclose(gb[on], z.imag[on])
    assert not got[1].any() and torch.allclose(got[on][..., 16:], y[on][..., 16:])


def test_rope_table():
    t = B.rope_table(100, 64, device="cpu")
    assert t.shape == (100, 64) and torch.equal(t, R.rope_table(100, 64)) or (
        t - R.rope_table(100, 64)).abs().max() < 1e-6
    for rotary in (0, 3, -2):
        with pytest.raises(ValueError):
            B.rope_table(10, rotary, device="cpu")


def test_workspace_sizes():
    f = B.lib().nvfp4_qk_norm_rope_workspace_bytes
    assert f(1, 1, 0, 16) >= 2 * 16 * 4
    assert 148 * 128 * 4 <= f(1 << 20, 32, 8, 128) <= 1 << 20
    for bad in ((0, 1, 1, 64), (1, 0, 1, 64), (1, 1, -1, 64), (1, 1, 1, 0), (1, 1, 1, 24), (1, 1, 1, 528),
                (1 << 31, 1, 1, 64), (1, 1 << 21, 1, 64)):
        assert f(*bad) == 0


def _forward(over):
    a = dict(q=0x10000, k=0x20000, hq=4, hk=2, q_strides=(512, 64), k_strides=(512, 64), in_dtype=1, T=10, D=64,
             qw=None, kw=None, eps=1e-6, positions=None, table=P, rows=10, rotary=64, q_out=0x30000,
             k_out=0x40000, out_strides=(256, 64), out_dtype=1, no_q=False, no_k=False)
    a.update(over)
    q = B.HeadsStruct(a["q"], a["hq"], *a["q_strides"])
    k = B.HeadsStruct(a["k"], a["hk"], *a["k_strides"])
    qo = B.HeadsStruct(a["q_out"], a["hq"], *a["out_strides"])
    ko = B.HeadsStruct(a["k_out"], a["hk"], *a["out_strides"])
    fwd = B.lib().nvfp4_qk_norm_rope(
        None if a["no_q"] else ctypes.byref(q), None if a["no_k"] else ctypes.byref(k), a["in_dtype"], a["T"],
        a["D"], a["qw"], a["kw"], a["eps"], a["positions"], a["table"], a["rows"], a["rotary"], 0,
        ctypes.byref(qo), ctypes.byref(ko), a["out_dtype"], None, None)
    bwd = B.lib().nvfp4_qk_norm_rope_backward(
        ctypes.byref(q), ctypes.byref(k), a["in_dtype"], None if a["no_q"] else ctypes.byref(q),
        None if a["no_k"] else ctypes.byref(k), a["in_dtype"], a["T"], a["D"], a["qw"], a["kw"], a["eps"],
        a["positions"], a["table"], a["rows"], a["rotary"], 0, ctypes.byref(qo), ctypes.byref(ko),
        a["out_dtype"], P, P, P, None, None)
    return fwd, bwd


BAD = ctypes.c_void_p(0x10008)


@pytest.mark.parametrize("over,expected", [
    (dict(no_q=True), B.ERR_NULL), (dict(q=None), B.ERR_NULL), (dict(k=None), B.ERR_NULL),
    (dict(q_out=None), B.ERR_NULL), (dict(k_out=None), B.ERR_NULL), (dict(table=None), B.ERR_NULL),
    (dict(in_dtype=2), B.ERR_ARG), (dict(out_dtype=-1), B.ERR_ARG),
    (dict(eps=0.0), B.ERR_ARG), (dict(eps=float("nan")), B.ERR_ARG), (dict(eps=float("inf")), B.ERR_ARG),
    (dict(eps=-1e-6), B.ERR_ARG),
    (dict(T=0), B.ERR_SHAPE), (dict(T=11), B.ERR_SHAPE), (dict(D=24), B.ERR_SHAPE),
    (dict(D=0), B.ERR_SHAPE), (dict(D=528), B.ERR_SHAPE), (dict(rotary=24), B.ERR_SHAPE),
    (dict(rotary=80), B.ERR_SHAPE), (dict(rotary=-16), B.ERR_SHAPE), (dict(rows=0), B.ERR_SHAPE),
    (dict(hq=0), B.ERR_SHAPE), (dict(hk=-1), B.ERR_SHAPE), (dict(q_strides=(-512, 64)), B.ERR_SHAPE),
    (dict(out_strides=(64, 64)), B.ERR_SHAPE), (dict(out_strides=(256, 0)), B.ERR_SHAPE),
    (dict(out_strides=(0, 64)), B.ERR_SHAPE), (dict(out_strides=(248, 64)), B.ERR_SHAPE),
    (dict(out_strides=(64, 632)), B.ERR_SHAPE), (dict(out_strides=(56, 640)), B.ERR_SHAPE),
    (dict(q_strides=(516, 64)), B.ERR_ALIGN), (dict(k_strides=(512, 68)), B.ERR_ALIGN),
    (dict(q=0x10008), B.ERR_ALIGN), (dict(k_out=0x40004), B.ERR_ALIGN), (dict(table=BAD), B.ERR_ALIGN),
    (dict(qw=BAD), B.ERR_ALIGN), (dict(kw=BAD), B.ERR_ALIGN),
    (dict(positions=ctypes.c_void_p(0x10002)), B.ERR_ALIGN)])
def test_head_refusals(over, expected):
    assert _forward(over) == (expected, expected)


@pytest.mark.skipif(torch.cuda.is_available(), reason="no work may be queued with these addresses")
@pytest.mark.parametrize("over", [
    dict(), dict(no_k=True), dict(hk=0, k=None, k_out=None), dict(rotary=0, table=None, rows=0),
    dict(out_strides=(64, 640)), dict(q_strides=(0, 0), k_strides=(8, 8)), dict(T=1, out_strides=(3, 64)),
    dict(positions=P, T=1000), dict(in_dtype=0, q_strides=(516, 68))])
def test_head_calls_that_are_accepted(over):
    """They get as far as looking for the GPU."""
    forward, backward = _forward(over)
    assert forward in (B.ERR_DEVICE, B.ERR_CUDA)
    assert backward in (B.ERR_DEVICE, B.ERR_CUDA)


def test_binding_refusals(monkeypatch):
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    table, p, w = torch.zeros(8, 64), torch.zeros(5, dtype=torch.int32), torch.ones(64)

    def both(error, match="", q=q, k=k, positions=p, table=table, q_weight=w, k_weight=w, **kw):
        with pytest.raises(error, match=match):
            B.qk_norm_rope(q, k, positions, table, q_weight, k_weight, **kw)
        with pytest.raises(error, match=match):
            B.qk_norm_rope_backward(q, k, q, k, positions, table, q_weight, k_weight, **kw)
    both(ValueError, "current CUDA device")
    both(TypeError, "q must be", q=q.half(), k=k.half())
    both(TypeError, "k must be", k=k.float())
    both(ValueError, "k must be", k=k[:4])
    both(ValueError, "k must be", k=k[..., :48])
    both(ValueError, "q must be", q=q[0])
    both(ValueError, "unit stride", q=torch.zeros(5, 4, 128, dtype=torch.bfloat16)[..., ::2])
    both(TypeError, "positions", positions=p.long())
    both(ValueError, "positions", positions=p[:4])
    both(TypeError, "table", table=table.double())
    both(ValueError, "table", table=table[:, ::2])
    both(ValueError, "table", table=table[0])
    both(TypeError, "q_weight", q_weight=w.bfloat16())
    both(ValueError, "k_weight", k_weight=w[:32])
    with pytest.raises(TypeError, match="k_out"):
        B.qk_norm_rope(q, k, p, table, w, w, q_out=torch.zeros(5, 4, 64), k_out=k)
    with pytest.raises(ValueError, match="q_out"):
        B.qk_norm_rope(q, k, p, table, w, w, q_out=q[:4])
    with pytest.raises(ValueError, match="dk must be given"):
        B.qk_norm_rope_backward(q, None, q, k, p, table)
    with pytest.raises(ValueError, match="workspace has"):
        B.qk_norm_rope_backward(q, k, q, k, p, table, workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        B.qk_norm_rope_backward(q, k, q, k, p, table,
                                workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 20))
    with pytest.raises(ValueError, match="dq_weight"):
        B.qk_norm_rope_backward(q, k, q, k, p, table, dq_weight=w[:32])
    if not torch.cuda.is_available():
        monkeypatch.setattr(B, "_queue", lambda *a: None)
        for call in (B.qk_norm_rope, lambda q, k, **kw: B.qk_norm_rope_backward(q, k, q, k, **kw)):
            with pytest.raises(TypeError, match="dev_status"):
                call(q, k, dev_status=torch.zeros(1))


# ---- orthogonalisation ---------------------------------------------------------------------

def test_orthogonalize_reference():
    """Singular vectors stay, singular values go through the polynomial of every step."""
    torch.manual_seed(0)
    for shape in ((5, 9), (9, 5), (6, 6)):
        g = torch.randn(shape).double()
        u, s, vt = torch.linalg.svd(g, full_matrices=False)
        s = s / (s.square().sum().sqrt() + 1e-7)
        for a, b, c in [R.MUON] * 5:
            s = a * s + b * s ** 3 + c * s ** 5
        assert torch.allclose(R.orthogonalize(g), (u * s) @ vt, atol=1e-12)
    g = torch.randn(50, 80).double()
    off = R.orthogonalize_rounded(g) - R.orthogonalize(g)
    assert 1e-4 < off.norm() / R.orthogonalize(g).norm() < 1e-2


def test_orthogonalize_workspace_sizes():
    f = B.lib().nvfp4_orthogonalize_workspace_bytes
    for batch, rows, cols in ((1, 1, 1), (3, 1000, 333), (32, 1408, 2048), (1, 20480, 5120), (65535, 16, 16)):
        m, n = sorted((rows, cols))
        pad = -(-m // 128) * -(-n // 128) * 128 * 128
        need = batch * (2 * pad + 2 * 2 * m * n + 2 * 2 * m * m + 2 * 4 * m)
        assert need <= f(batch, rows, cols) <= need + batch * (2 * 2 * 63 * m + 2 * 2 * 63 * m + 8 * 592 + 2 * 4 * 3) + 9 * 256
    for bad in ((0, 4, 4), (65536, 4, 4), (1, 0, 4), (1, 4, 0), (1, (1 << 18) + 1, 4), (1, 4, (1 << 18) + 1),
                (2, 1 << 18, 1 << 18), (-1, 4, 4)):
        assert f(*bad) == 0


def _orthogonalize(over):
    a = dict(G=0x10000, dtype=0, batch=2, rows=30, cols=50, ldg=50, gs=1500, steps=5, coef=R.MUON * 5, eps=1e-7,
             out=0x20000, ldo=50, os=1500, ws=P)
    a.update(over)
    coef = None if a["coef"] is None else (ctypes.c_float * len(a["coef"]))(*a["coef"])
    return B.lib().nvfp4_orthogonalize(
        a["G"], a["dtype"], a["batch"], a["rows"], a["cols"], a["ldg"], a["gs"], a["steps"], coef, a["eps"],
        a["out"], a["ldo"], a["os"], a["ws"], None, None)


@pytest.mark.parametrize("over,expected", [
    (dict(G=None), B.ERR_NULL), (dict(out=None), B.ERR_NULL), (dict(coef=None), B.ERR_NULL),
    (dict(ws=None), B.ERR_NULL), (dict(dtype=2), B.ERR_ARG), (dict(steps=0), B.ERR_ARG),
    (dict(steps=33, coef=R.MUON * 33), B.ERR_ARG), (dict(eps=-1.0), B.ERR_ARG),
    (dict(eps=float("nan")), B.ERR_ARG), (dict(eps=float("inf")), B.ERR_ARG),
    (dict(coef=R.MUON * 4 + (1.0, float("nan"), 1.0)), B.ERR_ARG),
    (dict(coef=(float("inf"), 0.0, 0.0) + R.MUON * 4), B.ERR_ARG),
    (dict(batch=0), B.ERR_SHAPE), (dict(rows=0), B.ERR_SHAPE), (dict(cols=0), B.ERR_SHAPE),
    (dict(rows=(1 << 18) + 1, os=1 << 30), B.ERR_SHAPE), (dict(ldg=-1), B.ERR_SHAPE),
    (dict(gs=-1), B.ERR_SHAPE), (dict(ldo=49), B.ERR_SHAPE), (dict(os=1499), B.ERR_SHAPE),
    (dict(os=0), B.ERR_SHAPE), (dict(G=0x10002), B.ERR_ALIGN), (dict(G=0x10001, dtype=1), B.ERR_ALIGN),
    (dict(out=0x20001), B.ERR_ALIGN), (dict(ws=BAD), B.ERR_ALIGN)])
def test_orthogonalize_refusals(over, expected):
    assert _orthogonalize(over) == expected


@pytest.mark.skipif(torch.cuda.is_available(), reason="no work may be queued with these addresses")
@pytest.mark.parametrize("over", [dict(), dict(ldg=0, gs=0), dict(ldg=7), dict(batch=1, gs=-5, os=-5),
                                  dict(batch=1, rows=1, ldg=-3, ldo=-3, gs=0, os=0), dict(eps=0.0),
                                  dict(G=0x10002, dtype=1, out=0x20002)])
def test_orthogonalize_calls_that_are_accepted(over):
    assert _orthogonalize(over) in (B.ERR_DEVICE, B.ERR_CUDA)


def test_orthogonalize_binding_refusals(monkeypatch):
    g = torch.zeros(2, 30, 50)
    out = torch.zeros(2, 30, 50, dtype=torch.bfloat16)
    for error, match, args in (
            (ValueError, "current CUDA device", dict()), (TypeError, "g must be", dict(g=g.double())),
            (ValueError, "g must be", dict(g=g[0, 0])), (ValueError, "g must be", dict(g=g[None])),
            (ValueError, "unit column stride", dict(g=g[..., ::2])), (ValueError, "steps", dict(steps=0)),
            (ValueError, "coefficients", dict(coefficients=(1.0, 2.0))),
            (ValueError, "coefficients", dict(coefficients=[R.MUON] * 4)),
            (ValueError, "coefficients", dict(coefficients=[(1.0, 2.0)] * 5)),
            (TypeError, "out must be", dict(out=out.float())), (ValueError, "out must be", dict(out=out[:1])),
            (ValueError, "unit column stride", dict(out=torch.zeros(2, 50, 30, dtype=torch.bfloat16).mT)),
            (B.NVFP4Error, "orthogonalize of", dict(g=g[:, :0])),
            (ValueError, "workspace has", dict(workspace=torch.zeros(8, dtype=torch.uint8))),
            (ValueError, "contiguous", dict(workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 24)))):
        args = dict(args)
        with pytest.raises(error, match=match):
            B.orthogonalize(args.pop("g", g), **args)
    if not torch.cuda.is_available():
        monkeypatch.setattr(B, "_queue", lambda *a: None)
        with pytest.raises(TypeError, match="dev_status"):
            B.orthogonalize(g, dev_status=torch.zeros(1))


@pytest.mark.parametrize("unit", ["qk_norm.cu", "orthogonalize.cu"])
def test_units_use_checked_accesses_only(unit):
    """Their arrays are reached through the checked loads, stores and copies only (read from the sources, since no
    call of a correct kernel can show a check that is missing)."""
    text = open(os.path.join(os.path.dirname(B.__file__), "csrc", unit)).read()
    code = re.sub(r"//[^\n]*", "", text)
    arrays = "g|x|rest|out|partials|addend|weight|dweight|positions|table|data"
    assert "__ldg(" not in code and "ld.global.nc" not in code
    assert not re.findall(rf"\b[ap]\.(?:{arrays})\s*\[(?!kind\]|0\]|1\]|i\])", code)
    assert not re.findall(rf"\*\s*[ap]\.(?:{arrays})\b(?!\s*\w)", code)
    assert not re.findall(r"st\.global|atomicAdd", code)
    assert len(re.findall(r"\bld\.global", code)) == (1 if unit == "orthogonalize.cu" else 0)  # load16, behind its check
