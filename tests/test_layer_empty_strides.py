"""Tensors without elements have no rows to lay out: any strides pass the binding's checks (CPU)."""
import pytest
import torch

from gated_convolution_sequence_amd import layer


@pytest.mark.parametrize("shape", [(0, 6), (3, 0, 6), (0, 5, 6), (4, 0)])
def test_an_expanded_tensor_of_no_elements(shape):
    t = torch.zeros(()).expand(shape)
    assert layer._row_stride(t, "t") is None
    assert layer._rows_like((t, t), ("t", "u"), t.shape, t.dtype, t.device) == shape[-1]


def test_elements_still_want_contiguous_rows():
    with pytest.raises(ValueError):
        layer._row_stride(torch.zeros(()).expand(3, 6), "t")
    with pytest.raises(ValueError):
        layer._row_stride(torch.zeros(6, 3).t(), "t")
    with pytest.raises(ValueError):
        layer._row_stride(torch.zeros(6).expand(3, 6), "t")
