"""Row strides as the operators take them: no GPU."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops


def test_a_single_rows_stride_says_nothing():
    """One token cut from a tensor of any row stride (the library wants multiples of 8 between rows)."""
    wide = torch.zeros(3, 4099, dtype=torch.bfloat16)
    for one in (wide[1:2, :256], torch.empty_strided((1, 256), (3, 1)), torch.empty(0, 256), wide[0, :256][None]):
        assert ops._rows(one, "x") == 256
    assert ops._rows(torch.zeros(1, 1)[:, :1], "x") == 1


def test_rows_apart():
    wide = torch.zeros(3, 4099)
    assert ops._rows(wide[:, :256], "x") == 4099
    assert ops._rows(wide[:2], "x") == 4099
    for bad in (wide.t(), wide[:, ::2], torch.zeros(1, 8).expand(4, 8)):
        with pytest.raises(ValueError):
            ops._rows(bad, "x")
