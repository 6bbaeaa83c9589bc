"""GPU parity of the head norms with the position rotation, forward and backward, against the
formulas in 64 bits; every test through both libraries."""
import pytest
import torch

import layer_ref as R
from nvfp4_testlib import need_gpu

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding

pytestmark = pytest.mark.gpu

U = 2.0 ** -24          # half a step of FP32
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
TINY = 2.0 ** -126      # below the normal range values come as subnormals or zero


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


def _cpu(*ts):
    return [None if t is None else t.cpu() for t in ts]


# Rounding of the forward pass, in half-steps: the sum of D squares 16 in a lane and 5 across lanes, the
# mean and eps 2, half of that in the root, the root 4, the two products 2: r x w is off by at most
# 18; the two products of the turn and their sum add 3.
FORWARD = 24


def _check_forward(z, x, w, eps, positions, table, interleaved, what):
    ref, size = R.qk(*_cpu(x, w), eps, *_cpu(positions, table), interleaved)
    got = z.double().cpu()
    tol = HALF[z.dtype] * ref.abs() * (1 + 2.0 ** -7) + FORWARD * U * size + TINY
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist())


# The gradient: dz turned back and times the weight 4, n 17; the mean of their products 4 + 17 + 1 + 21
# + 1, times n 18 more; the difference, the root (16) and two products: 24 for the first part of dx
# and 84 for the second.  dw: 22 for each product, and its sum 64 in a lane, 5 + 3 over heads and warps,
# 56 + 5 over the CTAs.
def _check_backward(dx, dw, d, x, w, eps, positions, table, interleaved, what):
    ref, dwr, (first, second, dsize) = R.qk_backward(*_cpu(d, x, w), eps, *_cpu(positions, table), interleaved)
    got = dx.double().cpu()
    tol = HALF[dx.dtype] * ref.abs() * (1 + 2.0 ** -7) + U * (24 * first + 84 * second) + TINY
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist())
    bad = ~((dw.double().cpu() - dwr).abs() <= (22 + 133) * U * dsize + TINY)
    assert not bad.any(), (what, "weight", torch.nonzero(bad)[:4].tolist())


def _inputs(T, Hq, Hk, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")
    qkv = (randn(T, Hq + 2 * Hk, D) * torch.exp(2 * randn(1, Hq + 2 * Hk, 1))).to(dtype)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    return q, k, 1 + 0.3 * randn(D), 1 + 0.3 * randn(D), randn


SHAPES = [  # T, Hq, Hk, D, rotary
    (1, 1, 1, 16, 16), (1, 32, 8, 128, 128), (3, 5, 2, 32, 16), (2, 3, 1, 48, 48), (7, 16, 4, 64, 64),
    (33, 40, 10, 80, 32), (5, 7, 3, 96, 96), (129, 32, 8, 128, 64), (4, 6, 2, 192, 64), (9, 4, 1, 256, 256),
    (2, 33, 17, 272, 16), (3, 2, 1, 512, 512), (1000, 4, 1, 128, 128), (2500, 3, 2, 64, 32)]


@pytest.mark.parametrize("T,Hq,Hk,D,rotary", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("x_type,z_type", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                           (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
def test_forward_and_backward(T, Hq, Hk, D, rotary, interleaved, x_type, z_type):
    q, k, qw, kw, randn = _inputs(T, Hq, Hk, D, x_type, T + D)
    table = B.rope_table(4096, rotary)
    assert torch.allclose(table.cpu(), R.rope_table(4096, rotary), rtol=0, atol=1e-6)
    p = torch.randint(0, 4096, (T,), device="cuda", dtype=torch.int32)
    if T > 2:
        p[T // 2] = -1
    st = _status()
    zq, zk = B.qk_norm_rope(q, k, p, table, qw, kw, eps=1e-5, interleaved=interleaved, out_dtype=z_type,
                            dev_status=st)
    assert zq.dtype == zk.dtype == z_type
    _check_forward(zq, q, qw, 1e-5, p, table, interleaved, "q")
    _check_forward(zk, k, kw, 1e-5, p, table, interleaved, "k")
    dq, dk = randn(T, Hq, D).to(z_type), randn(Hk, T, D).to(z_type).transpose(0, 1)
    for dx_type in (torch.bfloat16, torch.float32):
        gq, gk, wq, wk = B.qk_norm_rope_backward(dq, dk, q, k, p, table, qw, kw, eps=1e-5,
                                                 interleaved=interleaved, dx_dtype=dx_type, dev_status=st)
        assert gq.dtype == gk.dtype == dx_type
        _check_backward(gq, wq, dq, q, qw, 1e-5, p, table, interleaved, "dq")
        _check_backward(gk, wk, dk, k, kw, 1e-5, p, table, interleaved, "dk")
    assert int(st) == 0


def test_without_weights_positions_table_or_keys():
    q, k, qw, kw, randn = _inputs(37, 4, 2, 64, torch.bfloat16)
    table = B.rope_table(37, 64)
    d = randn(37, 4, 64).bfloat16()
    for args in (dict(table=table), dict(), dict(positions=torch.full((37,), -1, dtype=torch.int32,
                                                                        device="cuda")),
                 dict(table=table, q_weight=qw)):
        z, none = B.qk_norm_rope(q, None, **args)
        assert none is None
        _check_forward(z, q, args.get("q_weight"), 1e-6, args.get("positions"), args.get("table"), False, args)
        gq, gk, wq, wk = B.qk_norm_rope_backward(d, None, q, None, **args)
        assert gk is None and wk is None
        _check_backward(gq, wq, d, q, args.get("q_weight"), 1e-6, args.get("positions"), args.get("table"),
                        False, args)


def test_padding_is_not_looked_at_and_gives_zeros():
    T, Hq, Hk, D = 70, 6, 2, 80
    q, k, qw, kw, randn = _inputs(T, Hq, Hk, D, torch.bfloat16)
    table = B.rope_table(100, 32)
    p = torch.arange(T, dtype=torch.int32, device="cuda")
    p[50:], p[3] = -1, -2 ** 31
    pad = (p < 0).nonzero()[:, 0]
    clean = B.qk_norm_rope(q, k, p, table, qw, kw)
    dq, dk = randn(T, Hq, D).bfloat16(), randn(T, Hk, D).bfloat16()
    clean += B.qk_norm_rope_backward(dq, dk, q, k, p, table, qw, kw)
    for t in (q, k, dq, dk):
        t[pad] = float("nan")
    dirty = B.qk_norm_rope(q, k, p, table, qw, kw)
    dirty += B.qk_norm_rope_backward(dq, dk, q, k, p, table, qw, kw)
    for a, b in zip(clean, dirty):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    for z in dirty[:4]:
        assert not z[pad].any()


@pytest.mark.parametrize("where", [100, 101, 2 ** 31 - 1])
def test_a_position_beyond_the_table_is_reported(where):
    q, k, qw, kw, randn = _inputs(9, 2, 1, 64, torch.bfloat16)
    p = torch.arange(9, dtype=torch.int32, device="cuda")
    p[4] = where
    st = _status()
    zq, zk = B.qk_norm_rope(q, k, p, B.rope_table(100, 64), qw, kw, dev_status=st)
    assert int(st) == B.DEVSTAT_INDEX
    assert not zq[4].any() and not zk[4].any()
    _check_forward(zq, q, qw, 1e-6, p, B.rope_table(100, 64), False, "others")
    st.zero_()
    gq, gk, wq, wk = B.qk_norm_rope_backward(zq, zk, q, k, p, B.rope_table(100, 64), qw, kw, dev_status=st)
    assert int(st) == B.DEVSTAT_INDEX and not gq[4].any() and not gk[4].any()
    _check_backward(gq, wq, zq, q, qw, 1e-6, p, B.rope_table(100, 64), False, "others")


def test_heads_of_any_size():
    """Zero heads, values whose squares leave FP32 on either side, and NaN or Inf in one head."""
    q, k, qw, kw, randn = _inputs(6, 4, 2, 64, torch.float32)
    table = B.rope_table(6, 64)
    q[0, 0], q[1, 1] = 0, 0
    q[1], k[2] = q[1] * 1e30, k[2] * 1e36 / 20
    q[2] *= 1e-25
    zq, zk = B.qk_norm_rope(q, k, None, table, qw, kw, out_dtype=torch.float32)
    _check_forward(zq, q, qw, 1e-6, None, table, False, "q")
    _check_forward(zk, k, kw, 1e-6, None, table, False, "k")
    dq, dk = randn(6, 4, 64), randn(6, 2, 64)
    gq, gk, wq, wk = B.qk_norm_rope_backward(dq, dk, q, k, None, table, qw, kw, dx_dtype=torch.float32)
    _check_backward(gq, wq, dq, q, qw, 1e-6, None, table, False, "dq")
    _check_backward(gk, wk, dk, k, kw, 1e-6, None, table, False, "dk")
    for value in (float("nan"), float("inf")):
        bad = q.clone()
        bad[3, 2, 5] = value
        z, _ = B.qk_norm_rope(bad, k, None, table, qw, kw, out_dtype=torch.float32)
        assert torch.isnan(z[3, 2]).any()
        z[3, 2] = zq[3, 2]
        assert torch.equal(z, zq)


def test_outputs_in_place_and_inside_larger_buffers():
    T, Hq, Hk, D = 45, 8, 2, 128
    q, k, qw, kw, randn = _inputs(T, Hq, Hk, D, torch.bfloat16)
    table = B.rope_table(64, 128)
    zq, zk = B.qk_norm_rope(q, k, None, table, qw, kw)
    # rows of a wider matrix, of which nothing else changes
    wide = torch.full((T + 2, Hq + 2 * Hk + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    B.qk_norm_rope(q, k, None, table, qw, kw, q_out=wide[1:-1, :Hq], k_out=wide[1:-1, Hq:Hq + Hk])
    assert torch.equal(wide[1:-1, :Hq], zq) and torch.equal(wide[1:-1, Hq:Hq + Hk], zk)
    wide[1:-1, :Hq + Hk] = 7.0
    assert (wide == 7.0).all()
    # head by head, and heads apart
    hm = torch.full((Hq, T, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    B.qk_norm_rope(q, None, None, table, qw, q_out=hm[..., :D].transpose(0, 1))
    assert torch.equal(hm[..., :D].transpose(0, 1), zq) and (hm[..., D:] == 7.0).all()
    # in place
    dq, dk = randn(T, Hq, D).bfloat16(), randn(T, Hk, D).bfloat16()
    ref = B.qk_norm_rope_backward(dq, dk, q, k, None, table, qw, kw)
    x = torch.cat([q, k], 1).contiguous()
    got = B.qk_norm_rope_backward(dq, dk, x[:, :Hq], x[:, Hq:], None, table, qw, kw, dq_in=x[:, :Hq],
                                  dk_in=x[:, Hq:])
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    got = B.qk_norm_rope_backward(dq, dk, q, k, None, table, qw, kw, dq_in=dq, dk_in=dk)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    qkv = torch.cat([q, k, k], 1).contiguous()
    values = qkv[:, Hq + Hk:].clone()
    B.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], None, table, qw, kw, q_out=qkv[:, :Hq],
                   k_out=qkv[:, Hq:Hq + Hk])
    assert torch.equal(qkv[:, :Hq], zq) and torch.equal(qkv[:, Hq:Hq + Hk], zk)
    assert torch.equal(qkv[:, Hq + Hk:], values)


def test_heads_that_are_read_may_overlap():
    """A shared head, expanded: each of its copies has a gradient of its own."""
    q, k, qw, kw, randn = _inputs(12, 4, 1, 64, torch.bfloat16)
    table = B.rope_table(64, 64)
    shared = k.expand(12, 4, 64)
    zq, zk = B.qk_norm_rope(q, shared, None, table, qw, kw)
    _check_forward(zk, shared, kw, 1e-6, None, table, False, "shared")
    d = randn(12, 1, 64).bfloat16().expand(12, 4, 64)
    gq, gk, wq, wk = B.qk_norm_rope_backward(zq, d, q, shared, None, table, qw, kw)
    _check_backward(gk, wk, d, shared, kw, 1e-6, None, table, False, "shared")


def test_on_another_stream_and_replayed_for_other_positions():
    T = 300
    q, k, qw, kw, randn = _inputs(T, 8, 2, 128, torch.bfloat16)
    table = B.rope_table(2048, 128)
    p = torch.randint(0, 2048, (T,), device="cuda", dtype=torch.int32)
    dq, dk = randn(T, 8, 128).bfloat16(), randn(T, 2, 128).bfloat16()

    def both(stream=None):
        return (B.qk_norm_rope(q, k, p, table, qw, kw, stream=stream)
                + B.qk_norm_rope_backward(dq, dk, q, k, p, table, qw, kw, stream=stream))
    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, there))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both()
    for seed in range(3):
        torch.manual_seed(seed)
        p.copy_(torch.randint(-1, 2048, (T,), device="cuda", dtype=torch.int32))
        q.copy_(randn(T, 8, 128))
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, captured))
    del graph


def test_offsets_beyond_32_bits():
    """Heads further than 2^31 values apart."""
    far = torch.empty(2, (1 << 31) + 64, dtype=torch.bfloat16, device="cuda")
    x = far[:, :64][:, None]  # token stride 2^31 + 64
    x.copy_(torch.randn(2, 1, 64, device="cuda"))
    z = far[:, -64:][:, None]
    z.zero_()
    near = x.clone()
    B.qk_norm_rope(x, None, q_out=z)
    assert torch.equal(z, B.qk_norm_rope(near, None)[0])
    B.qk_norm_rope_backward(z, None, x, None, dq_in=z)
    want = B.qk_norm_rope_backward(B.qk_norm_rope(near, None)[0], None, near, None)[0]
    assert torch.equal(z, want)
