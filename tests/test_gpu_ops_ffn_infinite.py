"""An infinity in dy (a loss scale that overflows) reaches what it is a factor of, and nothing else of its expert."""
import math

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_ffn import GRAD_TOL, both, make, rel

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert F.fp8z1_ffn_timeouts() == 0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("token", [3, 200])
def test_columns_without_it_keep_their_sums(bad, token):
    """d_down = h^T dy: column j of it is a sum over dy's column j alone."""
    x, dy, w, off = make([260, 40], 304, 256, 7)
    clean = both(x, dy, w, off)
    dy[token, 18] = bad
    y, dx, d_gu, d_dn = both(x, dy, w, off)
    assert torch.equal(y, clean[0])
    others = [j for j in range(304) if j != 18]
    assert rel(d_dn[0][:, others], clean[3][0][:, others].double()) <= GRAD_TOL
    assert not d_dn[0][:, 18].isfinite().any()
    assert torch.equal(d_dn[1], clean[3][1]) and torch.equal(d_gu[1], clean[2][1])
    # dh of that token has no finite number, so neither has its dx, nor any sum over the expert's tokens
    assert not dx[token].isfinite().any() and not d_gu[0].isfinite().any()
    rest = [t for t in range(300) if t != token]
    assert torch.equal(dx[rest], clean[1][rest])
