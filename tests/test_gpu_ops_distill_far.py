"""The distillation loss where logits lie far from zero: a shift common to a row, masks of any finite value, teachers
near the type's limits."""
import math

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _ops as R
from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_distill import make

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

# A loss is the difference of p log p, p (z - m) / tau and log total.  Beside the maximum no number is above 30 (5 sigma of
# each side, and log of the vocabulary); about eight roundings of 2^-24 of that, and as much for exp2 and log: 3e-5.
LOSS_TOL = 3e-5


@pytest.mark.parametrize("tau", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("shift", [1000.0, -1000.0, 12345.678, 3.0e5, -1.0e7])
def test_common_shift(shift, tau):
    """The reference reads the same shifted FP32 logits, so that their own rounding is in both."""
    z, ids, t, w = make(6, 5000, 8, torch.float32, 11)
    z = z + shift
    if abs(shift) >= 1e7:
        z[:, 2500:] = 0.0  # and parts whose own maximum is far from the row's
        z[:, :2500] += abs(shift) * 2
    loss, d = ops.distill_loss_grad(z, ids, t, temperature=tau, row_weight=w)
    want, wd = R.distill(z, ids, t, tau, w)
    # a listed logit may lie 1e7 below the maximum: 2^-22 of what it adds to the loss
    assert ((loss.cpu().double() - want).abs() <= tau * tau * LOSS_TOL / min(tau, 1) + 2.0**-22 * want.abs()).all()
    size = w.cpu().double()[:, None] * tau
    q = wd / torch.where(size == 0, torch.ones_like(size), size)
    # (q - p) to 1e-5 of q + p, as without a shift
    assert ((d.cpu().double() - wd).abs() <= 1e-5 * (q.abs() + 2e-2) * size).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mask", [-1e4, -65504.0, -1e9, -1e12, -1e20, -1e30, 1e9, 1e12, 1e30])
def test_rows_of_nothing_but_a_mask(mask, dtype):
    """q is uniform; the loss is sum p log p + log vocab."""
    vocab = 3001
    z = torch.full((3, vocab), mask, device="cuda", dtype=dtype)
    z[1, 7] = z[1, 7] * 2 if mask < 0 else z[1, 7] / 2  # one far below
    z[2, :1500] = -math.inf
    ids = torch.tensor([[3, 5, 9]] * 3, dtype=torch.int32, device="cuda")
    ids[2] += 2000
    t = torch.tensor([[2.0, 1.0, 0.0]] * 3, device="cuda")
    loss, d = ops.distill_loss_grad(z, ids, t)
    want, wd = R.distill(z, ids, t, 1.0, None)
    assert ((loss.cpu().double() - want).abs() <= LOSS_TOL).all(), (loss, want)
    tol = 1e-5 * (wd.abs() + 2e-2) + (2.0**-8 * wd.abs() if dtype == torch.bfloat16 else 0)
    assert ((d.cpu().double() - wd).abs() <= tol).all()


def test_a_mask_beside_ordinary_logits():
    """Masked elements get nothing, whatever part of the row holds no other."""
    z, ids, t, w = make(8, 40_000, 8, torch.float32, 4)
    for r, mask in enumerate((-1e4, -1e6, -1e9, -1e12, -1e20, -1e30, torch.finfo(torch.float32).min, -math.inf)):
        z[r, 12_000:] = mask
    ids = torch.where(ids >= 12_000, ids % 12_000, ids)
    loss, d = ops.distill_loss_grad(z, ids, t, row_weight=w)
    want, wd = R.distill(z, ids, t, 1.0, w)
    assert ((loss.cpu().double() - want).abs() <= LOSS_TOL).all()
    assert (d[:, 12_000:] == 0).all()
    size = w.cpu().double()[:, None]
    q = wd / torch.where(size == 0, torch.ones_like(size), size)
    assert ((d.cpu().double() - wd).abs() <= 1e-5 * (q.abs() + 2e-2) * size).all()


def test_a_listed_id_masked_by_the_lowest_value():
    """Its loss is tau (m - z) p, within FP32 where (m - z) / tau is not."""
    lowest, tau = torch.finfo(torch.float32).min, 0.3
    z = torch.randn(2, 500, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    z[0, 7] = lowest
    ids = torch.tensor([[7, 3], [7, 3]], dtype=torch.int32, device="cuda")
    t = torch.tensor([[1.0, 1.0]] * 2, device="cuda")
    loss, d = ops.distill_loss_grad(z, ids, t, temperature=tau)
    want, wd = R.distill(z, ids, t, tau, None)
    assert want.isfinite().all() and want[0] > 1e37
    # the listed entries' p are 1/2 each: four roundings of 2^-23, and LOSS_TOL for the ordinary row
    assert ((loss.cpu().double() - want).abs() <= tau * tau * LOSS_TOL / tau + 2.0**-21 * want.abs()).all()
    assert ((d.cpu().double() - wd).abs() <= 1e-5 * tau * (wd.abs() / tau + 2e-2)).all()
