"""One token cut from a tensor whose row stride the kernels could not take."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_ffn import make

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


def test_one_token_of_an_odd_row_stride():
    x, dy, w, off = make([1], 256, 128, 2)
    want, saved = ops.ffn_forward(x, *w, offsets=off, save=True)
    grads = ops.ffn_backward(dy, x, saved, *w, offsets=off)
    wide = torch.zeros(2, 4099, dtype=torch.bfloat16, device="cuda")
    wide[0, :256], wide[0, 256:512] = x[0], dy[0]
    xs, dys, out = wide[:1, :256], wide[:1, 256:512], wide[:1, 512:768]
    y, saved = ops.ffn_forward(xs, *w, offsets=off, save=True, out=out)
    assert torch.equal(y, want) and y.data_ptr() == out.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(ops.ffn_backward(dys, xs, saved, *w, offsets=off), grads))
    assert not wide[1].any()
