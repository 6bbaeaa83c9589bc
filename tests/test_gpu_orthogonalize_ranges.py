"""The orthogonalisation at the ends of its range, against the steps in 64 bits; every test through both
libraries."""
import pytest
import torch

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
