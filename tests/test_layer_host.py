"""Host-side checks of the operators around a layer's products that need no GPU: the references against
differences, sizes, and refusals before any work is queued (C ABI and binding)."""
import ctypes

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
    assert f(1 << 20, 32, 8, 128) == 1776 * 128 * 4
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
