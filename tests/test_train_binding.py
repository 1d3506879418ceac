"""What the binding of the training-step operators passes on (CPU checks): row
pitches of views of which a stride says nothing."""
import pytest
import torch

from mxfp4_precision_numerics_amd import training

F = (torch.float32,)


def pitch(t, rows, cols):
    return training._rows("t", t, F, rows, cols)


def test_a_single_rows_stride_says_nothing():
    wide = torch.zeros(9, 33)
    assert pitch(wide[4:5, :32], 1, 32) == 32  # 33 would be refused for alignment
    assert pitch(wide[:, :32], 1, 32) == 32  # one row is addressed
    assert pitch(wide[:0, :32], 0, 32) == 32
    assert pitch(wide[::2, :32], 5, 32) == 66
    assert pitch(wide[:2, :32], 2, 32) == 33


def test_a_single_columns_stride_says_nothing():
    t = torch.zeros(1, 7).t()
    assert t.is_contiguous() and t.stride(1) != 1
    assert pitch(t, 7, 1) == 1
    with pytest.raises(ValueError, match="unit column stride"):
        pitch(torch.zeros(2, 7).t(), 7, 2)


@pytest.mark.parametrize("t,rows,cols", [(torch.zeros(3, 32), 4, 32), (torch.zeros(1, 31), 1, 32), (torch.zeros(0, 32), 1, 32)])
def test_a_view_too_small_is_refused(t, rows, cols):
    with pytest.raises(ValueError, match="the call addresses"):
        pitch(t, rows, cols)
