"""The step of a QKV projection with head norms, rotation and update, as the benchmark runs it: every operator
against its reference on what the one before gave, run again, captured and replayed."""
import pytest
import torch

import layer_ref as R
import synth
from nvfp4_testlib import need_gpu
from test_gpu_orthogonalize import _check as check_update
from test_gpu_qk_norm import _check_backward, _check_forward

pytest.importorskip("nvfp4_bit_quantized_03_b200")
import bench  # noqa: E402

pytestmark = pytest.mark.gpu


def _step():
    need_gpu()
    return bench.QKVStep(synth.QKVLayer("small", 3, 192, 320, 6, 2, 64), torch.device("cuda"))


def test_every_operator_of_the_step():
    step = _step()
    step.events = []
    out = step.run()
    torch.cuda.synchronize()
    assert int(step.dev_status) == 0
    assert [n for n, _, _ in step.events] == ["fprop", "norms", "norms backward", "dgrad", "wgrad", "update"]
    heads = out["qkv"].view(192, 10, 64)
    norm = 1e-6, step.positions, step.table, False
    _check_forward(out["q"], heads[:, :6], step.q_weight, *norm, "q")
    _check_forward(out["k"], heads[:, 6:8], step.k_weight, *norm, "k")
    _check_backward(out["dqkv"][:, :6], out["dq_weight"], step.dq, heads[:, :6], step.q_weight, *norm, "dq")
    _check_backward(out["dqkv"][:, 6:8], out["dk_weight"], step.dk, heads[:, 6:8], step.k_weight, *norm, "dk")
    assert torch.equal(out["dqkv"][:, 8:], step.dv)
    # the products are NVFP4 (checked against the oracle elsewhere): here only that they took these operands.  A
    # block's values are off by at most a sixth of its largest (half a step of 2 at 6, and the scale's 1/16) and,
    # rounded stochastically, by a third
    for got, want, size in ((out["qkv"].view(192, 640), step.x.double() @ step.w.double().T, 0.25),
                            (out["dw"], out["dqkv"].view(192, 640).double().T @ step.x.double(), 0.6)):
        assert (got.double() - want).norm() < size * want.norm()
    check_update(out["update"], out["dw"], "update")


def test_the_step_repeats_and_follows_its_inputs_in_a_graph():
    step = _step()
    first, again = step.run(), step.run()
    for name in first:
        assert torch.equal(first[name], again[name]), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step.run()
    for seed in range(2):
        torch.manual_seed(seed)
        step.x.copy_(torch.randn(192, 320, device="cuda"))
        step.dq.copy_(1e-3 * torch.randn(192, 6, 64, device="cuda"))
        step.positions.copy_(torch.randint(-1, 192, (192,), device="cuda", dtype=torch.int32))
        want = step.run()
        graph.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(want[name], captured[name]), (seed, name)
    assert int(step.dev_status) == 0
    del graph


def test_the_weight_gradients_of_a_layer_of_experts():
    """Each expert's matrix of experts_wgrad's output is orthogonalised by itself; one without tokens stays zero."""
    need_gpu()
    from nvfp4_bit_quantized_03_b200 import binding as B
    T, D, F, E = 300, 192, 256, 5
    g = torch.Generator(device="cuda").manual_seed(0)
    experts = torch.randint(0, 4, (T, 1), generator=g, device="cuda", dtype=torch.int32)  # none for the last one
    plan = B.expert_plan(experts, E)
    x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    dy = 1e-3 * torch.randn(plan.rows, F, generator=g, device="cuda").bfloat16()
    dw = B.experts_wgrad(dy, x, plan, 0x5A3C, 1, 0).view(E, F, D)
    update = B.orthogonalize(dw)
    assert dw[:4].any() and not dw[4].any() and not update[4].any()
    check_update(update[:4], dw[:4], "experts")
    for e in range(4):
        assert torch.equal(update[e], B.orthogonalize(dw[e]))
