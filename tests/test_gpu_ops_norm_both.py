"""The norm's result in 8 bits and in the rows' type from one pass: each as it is alone."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


# a warp a row and a CTA, 8 elements a thread and 32, whole 16 bytes and not
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 64), (700, 129), (40, 1000), (5000, 1024), (5000, 1001), (7, 7168), (1500, 7168),
                                      (900, 4097), (3, 16383), (0, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_both(residual, dtype, rows, dim):
    g = M.gen(rows + dim)
    x, r = (torch.randn(rows, dim, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(dim, generator=g, device="cuda") + 0.5
    r = r if residual else None
    y = ops.rms_norm(x, w, residual=r)
    codes, scale, *total = ops.rms_norm_fp8(x, w, residual=r)
    out = torch.empty_like(x)
    got = ops.rms_norm_fp8(x, w, residual=r, out=out)
    assert torch.equal(out, y[0] if residual else y)
    assert torch.equal(got[0].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(got[1], scale)
    assert len(got) == 2 + residual and all(torch.equal(a, b) for a, b in zip(got[2:], total))
    # rows of another stride, and in the input's place
    wide = M.strided(torch.zeros_like(x), 8)
    ops.rms_norm_fp8(x, w, residual=r, out=wide)
    assert torch.equal(wide, out)
    ops.rms_norm_fp8(x, w, residual=r, out=x)
    assert torch.equal(x, out)
