"""CPU checks of the 8-bit binding's view of torch tensors."""
import pytest
import torch

from nvfp4_bit_microscaled_amd import fp8


def test_row_stride():
    assert fp8._ld(torch.zeros(3, 5)) == 5
    assert fp8._ld(torch.zeros(3, 8)[:, :5]) == 8
    # a single row's stride is not used, and need not reach its width
    for t in (torch.zeros(5, 1).t(), torch.zeros(5)[None], torch.zeros(1, 5).as_strided((1, 5), (0, 1)),
              torch.zeros(5, 1).t().contiguous()):
        assert t.shape == (1, 5) and fp8._ld(t) == 5
    assert fp8._ld(torch.zeros(4, 8)[2:3, :5]) == 8
    assert fp8._ld(torch.zeros(0, 5)) == 5
    # nor is the step within rows of one element
    assert fp8._ld(torch.zeros(1, 3).t()) == 1 and fp8._ld(torch.zeros(3, 4)[:, 1:2]) == 4
    with pytest.raises(ValueError):
        fp8._ld(torch.zeros(5, 3).t())
    with pytest.raises(ValueError):
        fp8._ld(torch.zeros(1, 10)[:, ::2])
