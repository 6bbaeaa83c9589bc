"""Host-side checks of the binding's mixture-of-experts calls: strides, buffers and plans that it
accepts or refuses before a kernel is queued (no GPU needed)."""
import pytest
import torch

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding


@pytest.mark.parametrize("width", [64, 65, 4100])
def test_the_stride_of_a_single_row_does_not_matter(width):
    wide = torch.empty(3, width, dtype=torch.bfloat16)
    assert B._row_stride(wide[:1, :64]) == 64          # a slice of a wider buffer
    assert B._row_stride(wide[:1, :64].expand(1, 64)) == 64
    assert B._row_stride(torch.empty(64).expand(1, 64)) == 64
    assert B._row_stride(wide[:, :64]) == width        # with more rows it is the tensor's
    assert B._row_stride(wide[::2, :64]) == 2 * width


def test_a_workspace_whose_bytes_repeat_is_refused():
    """An expanded tensor has many elements and one byte behind them."""
    one = torch.zeros(1, dtype=torch.uint8).expand(1 << 24)
    experts = torch.zeros(2048, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        B.expert_plan(experts, 4, plan=B.ExpertPlan.empty(2048, 4, 4, device="cpu"), workspace=one)
    plan = B.ExpertPlan.empty(10, 2, 4, device="cpu")
    x = torch.zeros(plan.rows, 128, dtype=torch.bfloat16)
    W, Wt = (B.QuantizedTensor(*s, device="cpu") for s in ((4 * 128, 128), (128, 4 * 128)))
    for call in (lambda: B.quantize_grouped(x, plan, B.ROWWISE, workspace=one,
                                            out_row=B.QuantizedTensor(plan.rows, 128, device="cpu")),
                 lambda: B.experts_fprop(x, W, plan, gather=False, workspace=one),
                 lambda: B.experts_dgrad(x, Wt, plan, 0, 0, workspace=one),
                 lambda: B.experts_wgrad(x, x, plan, 0, 0, 0, gather=False, workspace=one)):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes host tensors as the device's")
@pytest.mark.parametrize("status", [torch.zeros(4, dtype=torch.uint8)[1:2],
                                    torch.zeros(1, dtype=torch.int64), torch.zeros(1),
                                    torch.zeros(0, dtype=torch.int32)])
def test_a_status_word_is_an_int32(monkeypatch, status):
    """A kernel writes four bytes there, on a 4-byte boundary."""
    monkeypatch.setattr(B, "_queue", lambda *a: None)  # the tensors here are the host's
    plan = B.ExpertPlan.empty(10, 2, 4, device="cpu")
    x, dw = torch.zeros(plan.rows, 128, dtype=torch.bfloat16), torch.zeros(10, 2)
    W, Wt = (B.QuantizedTensor(*s, device="cpu") for s in ((4 * 128, 128), (128, 4 * 128)))
    A, At = (B.QuantizedTensor(*s, device="cpu") for s in ((plan.rows, 128), (128, plan.rows)))
    experts, logits = torch.zeros(10, 2, dtype=torch.int32), torch.zeros(10, 4)
    for call in (lambda st: B.route(logits, 2, dev_status=st),
                 lambda st: B.route_backward(logits, experts, dw, dev_status=st),
                 lambda st: B.expert_plan(experts, 4, dev_status=st),
                 lambda st: B.quantize_grouped(x, plan, B.ROWWISE, out_row=A, dev_status=st),
                 lambda st: B.gemm_grouped(A, W, plan, dev_status=st),
                 lambda st: B.gemm_grouped_k(At, At, plan, dev_status=st),
                 lambda st: B.experts_fprop(x, W, plan, gather=False, dev_status=st),
                 lambda st: B.experts_dgrad(x, Wt, plan, 0, 0, dev_status=st),
                 lambda st: B.experts_wgrad(x, x, plan, 0, 0, 0, gather=False, dev_status=st),
                 lambda st: B.combine(x, plan, dev_status=st),
                 lambda st: B.combine_backward(torch.zeros(10, 128), x, plan, dw, dev_status=st)):
        with pytest.raises(TypeError, match="dev_status"):
            call(status)


def test_a_plans_tensors_cannot_be_replaced():
    """The calls use the addresses that the plan was made with: a replaced tensor would leave them
    reading memory that has been given back."""
    plan = B.ExpertPlan.empty(10, 2, 4, device="cpu")
    for name in ("offsets", "pair_row", "row_token", "tokens", "k", "experts", "rows", "ref"):
        with pytest.raises(AttributeError, match=name):
            setattr(plan, name, getattr(plan, name))
    plan.offsets.zero_()    # their contents are the caller's
    plan.note = "first layer"
    other = B.ExpertPlan(plan.offsets.clone(), plan.pair_row, plan.row_token)
    assert other._struct.offsets == other.offsets.data_ptr() != plan.offsets.data_ptr()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (64, 2, 4), (1000, 8, 64)])
@pytest.mark.parametrize("I,O", [(1024, 128), (64, 2048), (1088, 1024), (64, 128)])
def test_experts_workspaces_hold_what_the_calls_put_there(T, k, E, I, O):
    """Codes, scales and amax of every operand a call quantizes, and both arrays of partial maxima:
    fprop rows x I, dgrad rows x O, wgrad O x rows and I x rows."""
    rows = B.expert_rows(T, k, E)

    def operand(r, c):
        assert B.codes_bytes(r, c) == r * c // 2
        assert B.scales_bytes(r, c) == -(-r // 128) * 128 * (c // 16)
        return r * c // 2 + -(-r // 128) * 128 * (c // 16) + 4
    partials = B.workspace_bytes(rows, max(I, O))
    assert partials >= 2 * 4 * 148
    need = max(operand(rows, I), operand(rows, O), operand(O, rows) + operand(I, rows)) + partials
    have = B.lib().nvfp4_experts_workspace_bytes(T, k, E, rows, I, O)
    # every piece starts on a 256-byte boundary: less than 256 bytes of padding each
    assert need <= have < need + 7 * 256
    chunks = -(-T * k // 1024)
    plan = B.lib().nvfp4_expert_plan_workspace_bytes(T, k, E)
    assert plan == 0 if chunks == 1 else plan >= 4 * chunks * E
