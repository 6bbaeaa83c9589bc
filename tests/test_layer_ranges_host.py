"""Host-side checks of the operators around a layer's products at the ends of their arguments' ranges (no
GPU)."""
import pytest
import torch

from test_layer_host import B, _forward, _orthogonalize

far = pytest.mark.skipif(torch.cuda.is_available(), reason="no work may be queued with these addresses")


@pytest.mark.parametrize("over", [dict(ldo=1 << 39, os=1 << 39), dict(os=1 << 39), dict(ldg=1 << 39), dict(gs=1 << 39)])
def test_matrix_strides_that_no_memory_has(over):
    """2^39 values of 2 bytes is what a tensor map's stride cannot hold."""
    assert _orthogonalize({**dict(rows=30, cols=48), **over}) == B.ERR_SHAPE


@far
@pytest.mark.parametrize("over", [dict(ldo=1 << 33, os=1 << 38), dict(ldg=1 << 38, gs=1 << 38),
                                  dict(batch=1, gs=1 << 50, os=1 << 50), dict(batch=1, rows=1, ldg=1 << 50, ldo=1 << 50)])
def test_matrix_strides_that_are_accepted(over):
    assert _orthogonalize({**dict(rows=30, cols=48), **over}) in (B.ERR_DEVICE, B.ERR_CUDA)
