"""The gradient of the head norms at the ends of its range, against the formulas in 64 bits; every test
through both libraries."""
import pytest
import torch

import layer_ref as R
from nvfp4_testlib import need_gpu

nv = pytest.importorskip("nvfp4_bit_quantized_03_b200")
B = nv.binding

pytestmark = pytest.mark.gpu

U = 2.0 ** -24      # half a step of FP32
TINY = 2.0 ** -126  # below the normal range values come as subnormals or zero


@pytest.fixture(params=["release", "checked"], autouse=True)
def _library(request):
    need_gpu()
    if request.param == "release":
        yield
    else:
        with B.bounds_checked():
            yield


# In half-steps of FP32: the root 16 (21 for the sum of squares, 2 for mean and eps, of which half, and 4 of its
# own), dz turned back and times the weight 4, e = r dy 17 on top; n 17; the mean of their products 4 + 17 + 1 + 21 +
# 1, times r 17 and times n 18 more: 24 for dx's first part, 84 for its second.  dw: 22 for each product, and its sum
# 64 in a lane, 5 + 3 over heads and warps, 56 + 5 over the CTAs.
@pytest.mark.parametrize("size,gradient,eps", [(1e18, 1e-6, 1e-6), (1e17, 1e-6, 1e-6), (1e17, 1e-9, 1e-6),
                                               (1e16, 1e-9, 1e-6), (1e17, 1.0, 1e-6), (1e-14, 1e12, 1e-30),
                                               (1e-10, 1e15, 1e-30)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_far_from_their_heads_in_size(size, gradient, eps, interleaved):
    g = torch.Generator(device="cuda").manual_seed(7)
    T, H, D = 11, 5, 64
    x = size * torch.randn(T, H, D, generator=g, device="cuda")
    d = gradient * torch.randn(T, H, D, generator=g, device="cuda")
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    table = B.rope_table(T, 32)
    dx, _, dw, _ = B.qk_norm_rope_backward(d, None, x, None, None, table, w, eps=eps, interleaved=interleaved,
                                           dx_dtype=torch.float32)
    ref, dwr, (first, second, dsize) = R.qk_backward(d.cpu(), x.cpu(), w.cpu(), eps, None, table.cpu(), interleaved)
    tol = U * (ref.abs() * (1 + 2.0 ** -7) + 24 * first + 84 * second) + TINY
    off = (dx.double().cpu() - ref).abs()
    assert (off <= tol).all(), float((off / tol).max())
    assert ((dw.double().cpu() - dwr).abs() <= (22 + 133) * U * dsize + TINY).all()


@pytest.mark.parametrize("H,D", [(20, 64), (3, 128), (7, 32), (5, 80)])
@pytest.mark.parametrize("value,dtype", [(float("inf"), torch.bfloat16), (float("-inf"), torch.bfloat16),
                                         (float("inf"), torch.float32)])
def test_an_infinite_gradient_stays_with_its_value_of_the_weight(H, D, value, dtype):
    """In the last head, and in every head before it, of a token among so many that a warp takes all heads of one: lanes
    behind the last head have worked on another one before."""
    T = 2600
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    d = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    w = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    clean, _, dw_clean, _ = B.qk_norm_rope_backward(d, None, x, None, q_weight=w)
    for h in range(H):
        hit = d.clone()
        hit[100 * h, h, h + 3] = value
        dx, _, dw, _ = B.qk_norm_rope_backward(hit, None, x, None, q_weight=w)
        want = dw_clean.clone()
        want[h + 3] = value * float(x[100 * h, h, h + 3])
        assert torch.equal(dw, want), (h, dw[h + 3])
        dx[100 * h, h] = clean[100 * h, h]
        assert torch.equal(dx, clean)


def test_outputs_over_other_heads_are_refused():
    T, D = 40, 64
    buf = torch.randn(T, 12, D, device="cuda").bfloat16()
    q, k = buf[:, :4], buf[:, 4:8]
    table = B.rope_table(T, D)
    before = buf.clone()
    wide = buf.view(torch.float32)  # [T, 12, D / 2]

    def refused(f, *a, **kw):
        with pytest.raises(B.NVFP4Error) as e:
            f(*a, **kw)
        assert e.value.status == B.ERR_SHAPE
        torch.cuda.synchronize()
        assert torch.equal(buf, before)
    d = torch.randn(T, 4, D, device="cuda").bfloat16()
    for out in (k, buf[:, 3:7], buf[:, 1:5], buf.flatten()[:T * 4 * D].view(T, 4, D), buf[1:].flatten()[:T * 4 * D].view(T, 4, D)):
        refused(B.qk_norm_rope, q, k, None, table, q_out=out)
        refused(B.qk_norm_rope_backward, d, d, q, k, None, table, dq_in=out)
    refused(B.qk_norm_rope, q, k, None, table, q_out=buf[:, 8:], k_out=buf[:, 8:])
    refused(B.qk_norm_rope, q, k, None, table, k_out=q)
    refused(B.qk_norm_rope, q, q, None, table, k_out=q)  # read as queries too
    refused(B.qk_norm_rope_backward, q, k, d, d, None, table, dq_in=k, dk_in=q)
    two = torch.randn(T, 2, D, device="cuda").bfloat16()
    refused(B.qk_norm_rope, q[:, :2], None, None, table, q_out=wide.as_strided((T, 2, D), (12 * D // 2, D, 1)))
    refused(B.qk_norm_rope_backward, two, None, q[:, :2], None, None, table,
            dq_in=wide.as_strided((T, 2, D), (12 * D // 2, D, 1)))
    # beside them in the same rows, and in place
    B.qk_norm_rope(q, k, None, table, q_out=q, k_out=buf[:, 8:])
    B.qk_norm_rope_backward(d, buf[:, 8:], q, k, None, table, dq_in=d, dk_in=buf[:, 8:])
    assert torch.equal(buf[:, 4:8], before[:, 4:8]) and not torch.equal(buf[:, 8:], before[:, 8:])
