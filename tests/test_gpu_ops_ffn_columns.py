"""Weight gradients column by column: columns of small numbers keep FP32's accuracy beside large ones."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from tests import _ops as R
from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_ffn import GRAD_TOL, both, gen

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert F.fp8z1_ffn_timeouts() == 0


def quantize(w):
    """Codes and block scales of a weight [E, R, C]."""
    e, r, c = w.shape
    scale = torch.zeros(e, R.blocks(r), R.blocks(c), device="cuda")
    codes = torch.zeros(w.shape, dtype=torch.uint8, device="cuda")
    for i in range(scale.shape[1]):
        for j in range(scale.shape[2]):
            at = (slice(None), slice(i * 128, i * 128 + 128), slice(j * 128, j * 128 + 128))
            scale[:, i, j] = w[at].abs().amax((1, 2)) / 448
            codes[at] = (w[at] / scale[:, i, j][:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale


def make(counts, hidden, inner, gate0, up1=None):
    """Feature 0 of a token is 1 and drives gate column f by gate0[f] (and feature 1 up column f by up1[f]); the others
    are ordinary."""
    g = gen(hidden + inner + len(counts))
    e, n = len(counts), sum(counts)
    w = torch.randn(e, hidden, 2 * inner, generator=g, device="cuda") * hidden**-0.5
    w[:, :2] = 0
    w[:, 0, :inner] = gate0
    if up1 is not None:
        w[:, 1, inner:] = up1
    gu, gus = quantize(w)
    dn, dns = quantize(torch.randn(e, inner, hidden, generator=g, device="cuda") * inner**-0.5)
    x = torch.randn(n, hidden, generator=g, device="cuda")
    x[:, 0], x[:, 1] = 1, 0
    dy = torch.randn(n, hidden, generator=g, device="cuda").bfloat16()
    off = torch.tensor([sum(counts[:i]) for i in range(e + 1)], dtype=torch.int32, device="cuda")
    return x.bfloat16(), dy, (gu, gus, dn, dns), off


def worst(got, want, dim):
    """The largest error of a line of the gradient, relative to the line's norm, for each expert."""
    return ((got.double() - want).norm(dim=dim) / want.norm(dim=dim)).amax(0)


def reference(x, dy, w, off):
    return R.ffn(x, R.decode(w[0], w[1]), R.decode(w[2], w[3]), R.runs(off, w[0].shape[0], x.shape[0]), dy)


@pytest.mark.parametrize("counts,hidden,inner", [([300], 512, 256), ([40, 129, 0, 600], 272, 384), ([3, 1], 256, 128)])
def test_shut_gates(counts, hidden, inner):
    """Columns whose gate sits at -10, -20, -30 or -60 for every token, among open ones: silu is down to 1e-25 there."""
    level = torch.tensor([1.0, -10.0, -20.0, -30.0, -60.0], device="cuda")[torch.arange(inner, device="cuda") % 5]
    x, dy, w, off = make(counts, hidden, inner, level)
    _, _, d_gu, d_dn = both(x, dy, w, off)
    want = reference(x, dy, w, off)
    has = torch.tensor([n > 0 for n in counts], device="cuda")
    # an FP32 gate of size |g| is off by up to 32 units of 2^-24 |g| (sums over up to 512 terms), and exp(g) by that
    # much of itself
    tol = GRAD_TOL + level.abs().double() * 2.0**-19
    assert (worst(d_dn[has], want["d_down"][has], 2) <= tol).all()
    assert (worst(d_gu[has], want["d_gate_up"][has], 1) <= tol.repeat(2)).all()


def test_peaks_of_gate_and_up_in_different_tokens():
    """Gates of 4096 in one token, ups of 4096 in another, everything of size 1 in the rest."""
    x, dy, w, off = make([200, 70], 256, 256, torch.ones(256, device="cuda"), torch.ones(256, device="cuda"))
    x[5, 0], x[17, 1] = 4096, 4096
    x[5, 1] = x[17, 0] = 0
    dy[5] = dy[17] = 0  # neither is in the sums
    _, _, d_gu, d_dn = both(x, dy, w, off)
    want = reference(x, dy, w, off)
    assert (worst(d_dn, want["d_down"], 2) <= GRAD_TOL).all()
    assert (worst(d_gu, want["d_gate_up"], 1) <= GRAD_TOL).all()


def test_columns_of_every_size():
    """Up columns from 1e-12 to 1e12: every row of d_down and column of d_gate_up to its own accuracy."""
    x, dy, w, off = make([257, 30], 512, 512, torch.zeros(512, device="cuda"))
    size = torch.logspace(-12, 12, 4, device="cuda")  # the scale blocks' columns
    w[1][:, :, 4:] *= size
    _, _, d_gu, d_dn = both(x, dy, w, off)
    want = reference(x, dy, w, off)
    assert (worst(d_dn, want["d_down"], 2) <= GRAD_TOL).all()
    assert (worst(d_gu, want["d_gate_up"], 1) <= GRAD_TOL).all()
