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


@pytest.mark.parametrize("counts,hidden,inner", [([300], 512, 512), ([90, 0, 161], 1040, 384), ([40], 528, 2048)])
def test_h_and_dgu_are_held_finer_than_bf16(counts, hidden, inner):
    """One rounding to BF16 at the end (uniform errors: 2^-9.3 of the norm) and one of half that size before the second
    product: sqrt(1 + 1/4) 2^-9.3 = 2^-9.14 of the norm.  Two of BF16's would be 2^-8.8."""
    x, dy, w, off = make(counts, hidden, inner, 17)
    y, dx, _, _ = both(x, dy, w, off)
    want = R.ffn(x, R.decode(w[0], w[1]), R.decode(w[2], w[3]), R.runs(off, len(counts), x.shape[0]), dy)
    assert rel(y, want["y"]) <= 2.0**-9 and rel(dx, want["dx"]) <= 2.0**-9


def test_an_outlier_column_of_h():
    """One column of h far above the others: rows still carry BF16's accuracy of their own size."""
    x, dy, w, off = make([200], 512, 512, 18)
    w[1][:, :, 4] *= 1000  # the up columns of one scale block
    y, dx, _, _ = both(x, dy, w, off)
    want = R.ffn(x, R.decode(w[0], w[1]), R.decode(w[2], w[3]), R.runs(off, 1, 200), dy)
    for out, k in ((y, "y"), (dx, "dx")):
        assert ((out.double() - want[k]).norm(dim=1) <= 2.0**-8 * want[k].norm(dim=1)).all()


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
