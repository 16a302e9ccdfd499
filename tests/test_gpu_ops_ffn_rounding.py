"""What the roundings between the feed-forward products leave of y and dx."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from tests import _ops as R
from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_ffn import GRAD_TOL, both, make, rel

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert F.fp8z1_ffn_timeouts() == 0


@pytest.mark.parametrize("seed", [2, 39, 64, 94, 112])
def test_an_outlier_channel_of_x(seed):
    """A channel 300 times the others, in tokens of 1e-6 to 1e3: gates that nearly cancel hang on the small channels."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy, w, off = make([90, 200], 640, 256, 6)
    x *= torch.logspace(-6, 3, 290, device="cuda")[torch.randperm(290, generator=g, device="cuda")][:, None].bfloat16()
    dy *= torch.logspace(-3, 5, 290, device="cuda")[torch.randperm(290, generator=g, device="cuda")][:, None].bfloat16()
    x[:, 5] *= 300
    _, _, d_gu, d_dn = both(x, dy, w, off)
    want = R.ffn(x, R.decode(w[0], w[1]), R.decode(w[2], w[3]), R.runs(off, 2, 290), dy)
    assert rel(d_gu, want["d_gate_up"]) <= GRAD_TOL and rel(d_dn, want["d_down"]) <= GRAD_TOL
