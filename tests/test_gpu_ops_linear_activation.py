"""Activations of FP32 results where they are small: x is 0, so z is the bias and nothing else rounds."""
import math

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


# few rows, many; columns of whole 16 bytes, and not
@pytest.mark.parametrize("tokens", [3, 90, 3000])
@pytest.mark.parametrize("rows,cols,transposed", [(128, 4096, False), (4099, 128, True)])
@pytest.mark.parametrize("act,lo,hi", [("silu", -80.0, 80.0), ("gelu_tanh", -9.5, 10.0)])
def test_small_results_keep_their_bits(tokens, rows, cols, transposed, act, lo, hi):
    codes, scale = R.fp8_weight(M.gen(1), rows, cols)
    n = rows if transposed else cols
    z = torch.linspace(lo, hi, n, device="cuda")
    x = torch.zeros(tokens, cols if transposed else rows, dtype=torch.bfloat16, device="cuda")
    y, pre = ops.linear(x, codes, scale, bias=z, activation=act, transposed=transposed, dtype=torch.float32, save=True)
    assert torch.equal(pre, z.expand_as(pre))
    v = z.double()
    c = v if act == "silu" else math.sqrt(8 / math.pi) * (v + 0.044715 * v**3)
    want = v * torch.sigmoid(c)
    # z t / (1 + t), t = exp(-|c|), or z / (1 + t): t to 2 units of 2^-23, its sum half one, the division 2, the product half one:
    # less than 2^-20.  c of GELU: two constants and four operations, 6 of 2^-24 relative to c, and exp passes |c| times that on.
    tol = 2.0**-20 + (0 if act == "silu" else 6 * 2.0**-24 * c.abs())
    assert ((y.double() - want).abs() <= tol * want.abs() + 1e-44).all()


@pytest.mark.parametrize("tokens", [5, 700])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_same_bits_in_rows_of_any_stride(tokens, act, dtype):
    g = M.gen(tokens)
    codes, scale = R.fp8_weight(g, 256, 20480)
    x = torch.randn(tokens, 256, generator=g, device="cuda").bfloat16()
    y = ops.linear(x, codes, scale, activation=act, dtype=dtype)
    for pad, at in ((1, 0), (0, 1), (8, 0)):
        out = M.strided(torch.zeros_like(y), pad, at)
        assert torch.equal(ops.linear(x, codes, scale, activation=act, dtype=dtype, out=out), y)
