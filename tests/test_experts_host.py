"""Host-side checks of the mixture-of-experts entry points that need no GPU: sizes, and refusals
before any work is queued (through the C ABI and through the binding)."""
import ctypes

import numpy as np
import pytest
import torch

import experts_ref as R

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding

P = ctypes.c_void_p(0x10000)


def _plan(**over):
    v = dict(offsets=0x1000, pair_row=0x2000, row_token=0x3000, tokens=100, k=4, experts=8,
             rows=B.expert_rows(100, 4, 8))
    v.update(over)
    return B.PlanStruct(**v)


def _op(rows, cols, codes=0x10000, scales=0x20000, amax=0x30000):
    return B.Operand(codes, scales, amax, rows, cols)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 6, 64), (5, 3, 7), (128, 1, 1), (129, 2, 4),
                                   (1000, 8, 512), (16384, 8, 256)])
def test_expert_rows_is_the_worst_case(T, k, E):
    assert B.expert_rows(T, k, E) == R.expert_rows(T, k, E)
    assert B.expert_rows(T, k, E) % 128 == 0


@pytest.mark.parametrize("T,k,E", [(0, 1, 1), (-1, 1, 1), (1, 0, 1), (1, 33, 64), (1, 1, 0),
                                   (1, 1, 513), (1 << 31, 1, 1), (1 << 30, 4, 8), (1 << 23, 2, 8)])
def test_expert_rows_refuses_sizes_outside_the_limits(T, k, E):
    assert B.expert_rows(T, k, E) == 0


def test_every_routing_fits_its_rows():
    rng = np.random.default_rng(0)
    for _ in range(200):
        E = int(rng.integers(1, 20))
        k = int(rng.integers(1, E + 1))
        T = int(rng.integers(1, 300))
        counts = np.zeros(E, int)
        for _ in range(T):
            counts[rng.permutation(E)[:k]] += 1
        assert (-(-counts // 128) * 128).sum() <= B.expert_rows(T, k, E)


def test_workspace_sizes():
    assert B.lib().nvfp4_expert_plan_workspace_bytes(64, 8, 64) == 0        # one chunk of pairs
    assert B.lib().nvfp4_expert_plan_workspace_bytes(4096, 8, 64) >= 4 * 64 * 2
    rows = B.expert_rows(64, 2, 4)
    f = B.lib().nvfp4_experts_workspace_bytes
    need = max(B.codes_bytes(rows, 512) + B.scales_bytes(rows, 512),
               2 * B.codes_bytes(rows, 256) + 2 * B.scales_bytes(rows, 256))
    assert f(64, 2, 4, rows, 256, 256) >= need - rows * 256
    assert f(64, 2, 4, rows - 128, 256, 256) == 0
    assert f(64, 2, 4, rows, 32, 256) == 0 and f(64, 2, 4, rows, 64, 192) == 0


@pytest.mark.parametrize("over,expected", [
    (dict(logits=None), B.ERR_NULL), (dict(experts=None), B.ERR_NULL),
    (dict(weights=None), B.ERR_NULL), (dict(dtype=2), B.ERR_ARG), (dict(score=2), B.ERR_ARG),
    (dict(T=0), B.ERR_SHAPE), (dict(E=513, ld=513), B.ERR_SHAPE), (dict(k=0), B.ERR_SHAPE),
    (dict(k=33), B.ERR_SHAPE), (dict(k=17, E=16, ld=16), B.ERR_SHAPE), (dict(ld=63), B.ERR_SHAPE),
    (dict(groups=0), B.ERR_SHAPE), (dict(groups=33, E=66, ld=66), B.ERR_SHAPE),
    (dict(groups=3), B.ERR_SHAPE), (dict(groups=4, top=5), B.ERR_SHAPE),
    (dict(groups=4, top=0), B.ERR_SHAPE), (dict(groups=16, top=1, k=5), B.ERR_SHAPE),
    (dict(logits=ctypes.c_void_p(0x10002)), B.ERR_ALIGN),
    (dict(bias=ctypes.c_void_p(0x10002)), B.ERR_ALIGN)])
def test_route_refusals(over, expected):
    a = dict(logits=P, dtype=B.OUT_F32, T=10, E=64, ld=64, bias=None, score=0, groups=1, top=1, k=4,
             experts=P, weights=P)
    a.update(over)
    assert B.lib().nvfp4_route(a["logits"], a["dtype"], a["T"], a["E"], a["ld"], a["bias"],
                               a["score"], a["groups"], a["top"], a["k"], 1, 1.0, a["experts"],
                               a["weights"], None, None) == expected


@pytest.mark.parametrize("over,expected", [
    (dict(dweights=None), B.ERR_NULL), (dict(dlogits=None), B.ERR_NULL), (dict(ldd=63), B.ERR_SHAPE),
    (dict(score=-1), B.ERR_ARG), (dict(k=65), B.ERR_SHAPE),
    (dict(dlogits=ctypes.c_void_p(0x10001)), B.ERR_ALIGN)])
def test_route_backward_refusals(over, expected):
    a = dict(dtype=B.OUT_BF16, score=0, k=4, dweights=P, dlogits=P, ldd=64)
    a.update(over)
    assert B.lib().nvfp4_route_backward(P, a["dtype"], 10, 64, 64, P, a["dweights"], a["score"],
                                        a["k"], 1, 1.0, a["dlogits"], a["ldd"], None,
                                        None) == expected


PLAN_FAULTS = [
    (dict(offsets=None), B.ERR_NULL), (dict(pair_row=None), B.ERR_NULL),
    (dict(row_token=None), B.ERR_NULL), (dict(tokens=0), B.ERR_SHAPE), (dict(k=0), B.ERR_SHAPE),
    (dict(k=33), B.ERR_SHAPE), (dict(experts=0), B.ERR_SHAPE), (dict(experts=513), B.ERR_SHAPE),
    (dict(rows=128), B.ERR_SHAPE), (dict(rows=B.expert_rows(100, 4, 8) + 64), B.ERR_SHAPE),
    (dict(rows=128 * 65536), B.ERR_SHAPE), (dict(offsets=0x1002), B.ERR_ALIGN)]


@pytest.mark.parametrize("over,expected", PLAN_FAULTS)
def test_every_call_checks_its_plan(over, expected):
    L = B.lib()
    plan = ctypes.byref(_plan(**over))
    rows = over.get("rows", B.expert_rows(100, 4, 8))
    a, w = _op(rows, 256), _op(8 * 128, 256)
    ra, rw = ctypes.byref(a), ctypes.byref(w)
    col = ctypes.byref(_op(256, rows))
    assert L.nvfp4_plan_experts(P, plan, P, None, None) == expected
    assert L.nvfp4_quantize_grouped(P, 256, 256, plan, 0, B.ROWWISE, 0, 0, ra, None, P, None,
                                    None) == expected
    assert L.nvfp4_gemm_grouped(ra, rw, plan, P, 1, 128, None, None) == expected
    assert L.nvfp4_gemm_grouped_k(col, col, plan, P, 0, 256, None, None) == expected
    assert L.nvfp4_experts_fprop(P, 256, 1, rw, plan, 256, 128, P, 1, 128, P, None, None) == expected
    assert L.nvfp4_experts_dgrad(P, 128, ctypes.byref(_op(256, 8 * 128)), plan, 256, 128, 0, 0, P, 1,
                                 256, P, None, None) == expected
    assert L.nvfp4_experts_wgrad(P, 128, P, 256, 1, plan, 256, 128, 0, 0, 0, P, 0, 256, P, None,
                                 None) == expected
    assert L.nvfp4_combine(P, 256, 256, plan, P, P, 1, 256, None, None) == expected
    assert L.nvfp4_combine_backward(P, 1, 256, P, 256, 256, plan, P, P, 256, P, None,
                                    None) == expected
    assert L.nvfp4_combine(P, 256, 256, None, P, P, 1, 256, None, None) == B.ERR_NULL


def test_plan_needs_its_workspace_only_for_many_pairs():
    big = _plan(tokens=1024, k=8, experts=8, rows=B.expert_rows(1024, 8, 8))
    assert B.lib().nvfp4_plan_experts(P, ctypes.byref(big), None, None, None) == B.ERR_NULL
    assert B.lib().nvfp4_plan_experts(None, ctypes.byref(big), P, None, None) == B.ERR_NULL


@pytest.mark.parametrize("over,expected", [
    (dict(x=None), B.ERR_NULL), (dict(flags=B.SR), B.ERR_ARG),
    (dict(flags=B.ROWWISE | B.BLOCK2D), B.ERR_ARG), (dict(flags=B.ROWWISE | B.MX), B.ERR_ARG),
    (dict(flags=B.ROWWISE | 128), B.ERR_ARG), (dict(cols=264, ld=264), B.ERR_SHAPE),
    (dict(cols=272, ld=272), B.ERR_SHAPE), (dict(ld=248), B.ERR_SHAPE), (dict(ld=260), B.ERR_ALIGN),
    (dict(x=ctypes.c_void_p(0x10008)), B.ERR_ALIGN), (dict(ws=None), B.ERR_NULL),
    (dict(ws=ctypes.c_void_p(0x10008)), B.ERR_ALIGN), (dict(out=None), B.ERR_NULL),
    (dict(out=_op(128, 256)), B.ERR_SHAPE)])
def test_quantize_grouped_refusals(over, expected):
    a = dict(x=P, cols=256, ld=256, flags=B.ROWWISE, ws=P, out=_op(B.expert_rows(100, 4, 8), 256))
    a.update(over)
    out = ctypes.byref(a["out"]) if a["out"] is not None else None
    assert B.lib().nvfp4_quantize_grouped(a["x"], a["cols"], a["ld"], ctypes.byref(_plan()), 0,
                                          a["flags"], 0, 0, out, None, a["ws"], None,
                                          None) == expected


def test_grouped_flag_is_refused_elsewhere():
    out = _op(256, 512)
    assert B.lib().nvfp4_quantize(P, 256, 512, 512, B.ROWWISE | B.GATHER, 0, 0, ctypes.byref(out),
                                  None, P, None, None) == B.ERR_ARG


@pytest.mark.parametrize("a,b,dtype,ldd,expected", [
    ((0, 256), (8 * 128, 256), 1, 128, B.ERR_SHAPE),          # A has other rows
    (("rows", 256), (8 * 128, 320), 1, 128, B.ERR_SHAPE),     # K differs
    (("rows", 256), (8 * 64, 256), 1, 64, B.ERR_SHAPE),       # N not a multiple of 128
    (("rows", 96), (8 * 128, 96), 1, 128, B.ERR_SHAPE),       # K not a multiple of 64
    (("rows", 256), (120, 8 * 256), 1, 120, B.ERR_SHAPE),     # N not a multiple of 16
    (("rows", 256), (8 * 128, 256), 2, 128, B.ERR_ARG),
    (("rows", 256), (8 * 128, 256), 1, 112, B.ERR_SHAPE),
    (("rows", 256), (8 * 128, 256), 1, 132, B.ERR_ALIGN)])
def test_gemm_grouped_refusals(a, b, dtype, ldd, expected):
    rows = B.expert_rows(100, 4, 8)
    A, W = _op(rows if a[0] == "rows" else 128, a[1]), _op(*b)
    assert B.lib().nvfp4_gemm_grouped(ctypes.byref(A), ctypes.byref(W), ctypes.byref(_plan()), P,
                                      dtype, ldd, None, None) == expected


@pytest.mark.parametrize("m,n,rows_off,expected", [
    (64, 256, 0, B.ERR_SHAPE), (192, 256, 0, B.ERR_SHAPE), (128, 24, 0, B.ERR_SHAPE),
    (128, 256, 128, B.ERR_SHAPE), (1 << 29, 256, 0, B.ERR_SHAPE)])
def test_gemm_grouped_k_refusals(m, n, rows_off, expected):
    rows = B.expert_rows(100, 4, 8)
    A, W = _op(m, rows), _op(n, rows + rows_off)
    assert B.lib().nvfp4_gemm_grouped_k(ctypes.byref(A), ctypes.byref(W), ctypes.byref(_plan()), P,
                                        0, n, None, None) == expected


@pytest.mark.parametrize("I,O,expected", [(32, 128, B.ERR_SHAPE), (96, 128, B.ERR_SHAPE),
                                          (256, 192, B.ERR_SHAPE), (256, 0, B.ERR_SHAPE),
                                          (256, 1 << 28, B.ERR_SHAPE)])
def test_expert_linear_refusals(I, O, expected):
    L, plan = B.lib(), ctypes.byref(_plan())
    W, Wt = _op(8 * O, I), _op(I, 8 * O)
    assert L.nvfp4_experts_fprop(P, I, 1, ctypes.byref(W), plan, I, O, P, 1, O, P, None,
                                 None) == expected
    assert L.nvfp4_experts_dgrad(P, O, ctypes.byref(Wt), plan, I, O, 0, 0, P, 1, I, P, None,
                                 None) == expected
    assert L.nvfp4_experts_wgrad(P, O, P, I, 1, plan, I, O, 0, 0, 0, P, 0, I, P, None,
                                 None) == expected


@pytest.mark.parametrize("over,expected", [
    (dict(cols=4), B.ERR_SHAPE), (dict(cols=260), B.ERR_SHAPE), (dict(ldy=248), B.ERR_SHAPE),
    (dict(ldy=260), B.ERR_ALIGN), (dict(dtype=3), B.ERR_ARG), (dict(y=None), B.ERR_NULL),
    (dict(ldo=252), B.ERR_SHAPE), (dict(ldo=260), B.ERR_ALIGN), (dict(out=None), B.ERR_NULL)])
def test_combine_refusals(over, expected):
    a = dict(y=P, cols=256, ldy=256, out=P, dtype=B.OUT_BF16, ldo=256)
    a.update(over)
    plan = ctypes.byref(_plan())
    assert B.lib().nvfp4_combine(a["y"], a["cols"], a["ldy"], plan, P, a["out"], a["dtype"],
                                 a["ldo"], None, None) == expected
    assert B.lib().nvfp4_combine_backward(a["out"], a["dtype"], a["ldo"], a["y"], a["cols"],
                                          a["ldy"], plan, P, P, 256, P, None, None) == expected


def test_combine_backward_needs_its_weights():
    plan = ctypes.byref(_plan())
    assert B.lib().nvfp4_combine_backward(P, 1, 256, P, 256, 256, plan, None, P, 256, P, None,
                                          None) == B.ERR_NULL
    assert B.lib().nvfp4_combine_backward(P, 1, 256, P, 256, 256, plan, P, P, 256, None, None,
                                          None) == B.ERR_NULL


def test_binding_refuses_wrong_tensors_before_calling():
    plan = B.ExpertPlan.empty(10, 2, 4, device="cpu")
    with pytest.raises(ValueError):  # host tensors
        B.route(torch.zeros(10, 4), 2)
    with pytest.raises(TypeError):
        B.route(torch.zeros(10, 4, dtype=torch.float16), 2)
    with pytest.raises(ValueError):
        B.route(torch.zeros(4, 10).t(), 2)
    with pytest.raises(ValueError):
        B.route(torch.zeros(10, 4), 2, bias=torch.zeros(5))
    with pytest.raises(TypeError):
        B.expert_plan(torch.zeros(10, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        B.expert_plan(torch.zeros(9, 2, dtype=torch.int32), 4, plan=plan)
    with pytest.raises(ValueError):
        B.ExpertPlan(plan.offsets, plan.pair_row.t(), plan.row_token)
    with pytest.raises(B.NVFP4Error):
        B.ExpertPlan.empty(10, 33, 64, device="cpu")
    y = torch.zeros(plan.rows, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        B.combine(y.float(), plan)
    with pytest.raises(ValueError):
        B.combine(y[:64], plan)
    with pytest.raises(TypeError):
        B.combine(y, plan, torch.zeros(10, 2, dtype=torch.bfloat16))
    with pytest.raises(ValueError):  # all right, but on the host
        B.combine(y, plan, torch.zeros(10, 2))
    with pytest.raises(ValueError):
        B.combine_backward(torch.zeros(9, 64), y, plan, torch.zeros(10, 2))
    W = B.QuantizedTensor(4 * 128, 64, device="cpu")
    with pytest.raises(ValueError):  # rows of the tokens expected
        B.experts_fprop(y, W, plan)
    with pytest.raises(ValueError):
        B.experts_fprop(torch.zeros(10, 64, dtype=torch.bfloat16), W, plan,
                        workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.QuantizedTensor.from_buffers(W.codes, W.scales[:-1], W.amax)
    with pytest.raises(ValueError):
        B.QuantizedTensor.from_buffers(W.codes.t(), W.scales, W.amax)
    with pytest.raises(ValueError):  # one device
        B.QuantizedTensor.from_buffers(W.codes, W.scales, W.amax.to("meta"))
    with pytest.raises(ValueError):
        B.ExpertPlan(plan.offsets, plan.pair_row, plan.row_token.to("meta"))
    big = torch.zeros(2048, 4, dtype=torch.int32)
    with pytest.raises(ValueError):  # workspaces too small
        B.expert_plan(big, 4, plan=B.ExpertPlan.empty(2048, 4, 4, device="cpu"),
                      workspace=torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        B.quantize_grouped(y, plan, B.ROWWISE, workspace=torch.zeros(16, dtype=torch.uint8),
                           out_row=B.QuantizedTensor(plan.rows, 64, device="cpu"))
    q = B.QuantizedTensor.from_buffers(W.codes, W.scales, W.amax)
    assert (q.rows, q.cols) == (W.rows, W.cols)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_fail_cleanly():
    L, plan = B.lib(), ctypes.byref(_plan())
    bad = (B.ERR_CUDA, B.ERR_DEVICE)
    assert L.nvfp4_route(P, 0, 10, 64, 64, None, 0, 1, 1, 4, 1, 1.0, P, P, None, None) in bad
    assert L.nvfp4_plan_experts(P, plan, None, None, None) in bad
    assert L.nvfp4_combine(P, 256, 256, plan, None, P, 1, 256, None, None) in bad
    W = _op(8 * 128, 256)
    assert L.nvfp4_experts_fprop(P, 256, 1, ctypes.byref(W), plan, 256, 128, P, 1, 128, P, None,
                                 None) in bad
