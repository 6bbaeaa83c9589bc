"""Host-side checks of the operators around a layer's products at the ends of their arguments' ranges (no
GPU)."""
import pytest
import torch

from test_layer_host import B, P, _forward, _orthogonalize

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


@pytest.mark.parametrize("over", [
    # token 1's first head is token 0's third: what lies between the tokens, in values, passes 2^63
    dict(T=1 << 30, positions=P, out_strides=(1 << 34, 1 << 33)),
    dict(T=1 << 30, positions=P, out_strides=(1 << 38, 64)), dict(T=1 << 30, positions=P, q_strides=(1 << 38, 64)),
    dict(T=1 << 20, positions=P, k_strides=(1 << 32, 64)), dict(out_strides=(1 << 39, 64)),
    dict(out_strides=(64, 1 << 39)), dict(hq=1 << 20, out_strides=(1 << 20, 1 << 36))])
def test_head_strides_that_no_memory_has(over):
    assert _forward(over) == (B.ERR_SHAPE, B.ERR_SHAPE)


@far
@pytest.mark.parametrize("over", [dict(T=1 << 20, positions=P, out_strides=(1 << 28, 64)),
                                  dict(q_strides=(1 << 38, 1 << 37), out_strides=(1 << 38, 1 << 30))])
def test_head_strides_that_are_accepted(over):
    assert all(st in (B.ERR_DEVICE, B.ERR_CUDA) for st in _forward(over))
