"""Teacher logits near the type's limits: their quotient by a temperature below 1 leaves FP32, their differences do not."""
import math

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

LOWEST, LARGEST = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max


@pytest.mark.parametrize("tau", [0.25, 0.5, 1.0, 2.0])
@pytest.mark.parametrize("teacher", [
    [LOWEST, LOWEST, LOWEST],           # every entry masked alike: p is uniform
    [LOWEST, -math.inf, LOWEST],
    [3.0, LOWEST, 1.0],                 # masked entries beside ordinary ones
    [LARGEST, LARGEST, 0.0],
    [LARGEST, LOWEST, LOWEST],
])
def test_lowest_and_largest_values(teacher, tau):
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(1, 600, generator=g, device="cuda")
    ids = torch.tensor([[3, 590, 77]], dtype=torch.int32, device="cuda")
    t = torch.tensor([teacher], device="cuda")
    loss, d = ops.distill_loss_grad(z, ids, t, temperature=tau)
    want, wd = R.distill(z, ids, t, tau, None)
    assert want.isfinite().all()
    # numbers up to 30 / tau, about eight roundings of 2^-24
    assert abs(float(loss[0]) - float(want[0])) <= tau * tau * 3e-5 / min(tau, 1)
    assert ((d.cpu().double() - wd).abs() <= 1e-5 * tau * (wd.abs() / tau + 2e-2)).all()
