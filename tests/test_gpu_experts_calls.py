"""Calls of the mixture-of-experts operators that their documentation allows and that lie at the edge
of it: single rows out of wider buffers, and the like.  Through both libraries."""
import numpy as np
import pytest
import torch

import experts_ref as R
import synth
from nvfp4_testlib import need_gpu, to_device_bf16

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


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _row_of(t, width):
    """The one row of t as a slice of a buffer whose rows are `width` values."""
    wide = torch.zeros(1, width, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def test_one_token_out_of_a_wider_buffer():
    """Decoding: the token's row is a slice of a buffer of odd width, in every argument that has one."""
    st = _status()
    E, k, C = 6, 2, 256
    x = to_device_bf16(synth.activations((1, C), seed=1))
    logits = torch.from_numpy(np.random.default_rng(2).normal(0, 1, (1, E)).astype(np.float32)).cuda()
    w, _ = B.quantize(to_device_bf16(synth.weights((E * C, C), seed=3)), B.ROWWISE | B.BLOCK2D)

    def run(cut):
        l = cut(logits)
        e, wt = B.route(l, k, dev_status=st)
        plan = B.expert_plan(e, E, dev_status=st)
        q, _ = B.quantize_grouped(cut(x), plan, B.ROWWISE | B.GATHER, dev_status=st)
        y = B.experts_fprop(cut(x), w, plan, dev_status=st)
        out = B.combine(y, plan, wt, out=cut(torch.zeros(1, C, device="cuda")), dev_status=st)
        used = int(plan.offsets[-1])
        y[used:] = 0
        dy, dw = B.combine_backward(cut(out), y, plan, wt, dev_status=st)
        dy[used:] = 0
        dx = B.experts_wgrad(dy, cut(x), plan, 3, 1, 0, dev_status=st)
        dl = B.route_backward(l, e, dw, dlogits=cut(torch.zeros(1, E, device="cuda")), dev_status=st)
        return e, wt, q.codes[:used], y, out, dy, dw, dx, dl

    plain = run(lambda t: t)
    for got, ref in zip(run(lambda t: _row_of(t, t.shape[1] + 5)), plain):
        assert torch.equal(got, ref)
    assert int(st) == 0


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 3])
def test_the_router_takes_the_most_tokens(T):
    """Token counts up to the documented limit; the ends of the outputs against FP64."""
    logits = torch.full((T, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    ends = (slice(0, 1000), slice(T - 1000, T))
    for at in ends:
        logits[at, 0] = torch.linspace(-4, 4, 1000, device="cuda").bfloat16()
    st = _status()
    e, w = B.route(logits, 1, sigmoid=True, renorm=False, dev_status=st)
    assert not e.any()
    dl = B.route_backward(logits, e, w, sigmoid=True, renorm=False, dev_status=st)
    for at in ends:
        s = torch.sigmoid(logits[at].double())
        # exp to 2 units of 2^-23 and one rounding each of the sum and the quotient
        assert ((w[at].double() - s).abs() <= 8 * 2.0 ** -24 * s).all()
        # three such factors and their products, rounded to bf16
        ref = s * s * (1 - s)
        assert ((dl[at].double() - ref).abs() <= (2.0 ** -8 + 40 * 2.0 ** -24) * ref).all()
    middle = float(torch.sigmoid(torch.tensor(0.5, dtype=torch.float64)))
    low, high = torch.aminmax(w[1000:T - 1000])
    assert abs(float(low) - middle) <= 8 * 2.0 ** -24 and abs(float(high) - middle) <= 8 * 2.0 ** -24
    assert int(st) == 0


@pytest.mark.parametrize("T,k,E,I,O", [(50, 2, 4, 1088, 128), (50, 2, 4, 64, 1024),
                                       (5000, 4, 24, 320, 256)])
def test_calls_stay_inside_their_workspaces(T, k, E, I, O):
    """What lies behind a workspace of the documented size is left as it was."""
    guards = []

    def workspace(need):
        w = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        guards.append(w[need:])
        return w[:need] if need else None
    rng = np.random.default_rng(T)
    experts = torch.from_numpy(R.routing(rng, T, E, k)).cuda()
    plan = B.expert_plan(experts, E, workspace=workspace(
        B.lib().nvfp4_expert_plan_workspace_bytes(T, k, E)))
    x, xe, dy = (to_device_bf16(synth.activations(s, seed=1))
                 for s in ((T, I), (plan.rows, I), (plan.rows, O)))
    w = B.quantize(to_device_bf16(synth.weights((E * O, I), seed=2)),
                   B.ROWWISE | B.COLWISE | B.BLOCK2D)
    need = B.experts_workspace_bytes(plan, I, O)
    both = B.ROWWISE | B.COLWISE
    for flags in (B.ROWWISE, B.COLWISE, both, both | B.SR):
        B.quantize_grouped(xe, plan, flags, sign_mask=3,
                           workspace=workspace(B.workspace_bytes(plan.rows, I, flags)))
    for gather, a in ((True, x), (False, xe)):
        B.experts_fprop(a, w[0], plan, gather=gather, workspace=workspace(need))
        B.experts_wgrad(dy, a, plan, 5, 1, 0, gather=gather, workspace=workspace(need))
    B.experts_dgrad(dy, w[1], plan, 1, 0, workspace=workspace(need))
    torch.cuda.synchronize()
    for g in guards:
        assert (g == 0xA5).all()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_scores_that_fp64_cannot_tell_apart(sigmoid):
    """Without a bias or groups the logits are compared, with either the scores: sigmoids of 40 and 50
    are both 1 in FP64, softmax scores 800 below the largest both 0."""
    l = torch.tensor([[40.0, 50.0, 40.0, -3.0], [50.0, 40.0, 50.0, -3.0], [0.0, -800.0, -790.0, -810.0]],
                     device="cuda")
    by_logit = [[1, 0, 2], [0, 2, 1], [0, 2, 1]]
    if sigmoid:
        by_score = [[0, 1, 2], [0, 1, 2], [0, 1, 2]]
    else:        # exp(-10) it can, exp(-790) it cannot
        by_score = [[1, 0, 2], [0, 2, 1], [0, 1, 2]]
    st = _status()
    e, _ = B.route(l, 3, sigmoid=sigmoid, dev_status=st)
    assert e.tolist() == by_logit
    e, _ = B.route(l, 3, sigmoid=sigmoid, bias=torch.zeros(4, device="cuda"), dev_status=st)
    assert e.tolist() == by_score
    e, _ = B.route(l, 3, sigmoid=sigmoid, groups=2, top_groups=2, dev_status=st)
    assert e.tolist() == by_score
    assert int(st) == 0
