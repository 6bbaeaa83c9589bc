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
