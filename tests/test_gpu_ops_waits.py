"""Waits between the feed-forward kernels' warps that run out: what they belong to is NaN, the rest is whole, and the
device goes on.  The checked library leaves a kernel's first sums unannounced for it; its waits give up after 0.2 s."""
import os
import subprocess
import sys

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import build as fp8build
from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_ffn import both, make

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GATE_UP, DOWN, DH, DX, PART, D_DOWN, D_GATE_UP = (1 << i for i in range(7))


def test_on_the_checked_build(lib):
    if F.CHECKED:
        pytest.skip("runs the checked build from the release one")
    fp8build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_gpu_ops_waits.py::test_what_a_wait_belongs_to_is_nan"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, FP8Z1_CHECKED="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout and " skipped" not in r.stdout


# the outputs (y, dx, d_gate_up, d_down) that a kernel's sums reach
@pytest.mark.parametrize("kernel,reached", [
    (GATE_UP, (True, True, True, True)), (DOWN, (True, False, False, False)), (DH, (False, True, True, False)),
    (DX, (False, True, False, False)), (PART, (True, False, False, False)), (D_DOWN, (False, False, False, True)),
    (D_GATE_UP, (False, False, True, False))])
def test_what_a_wait_belongs_to_is_nan(lib, kernel, reached):
    if not F.CHECKED:
        pytest.skip("needs the checked build (FP8Z1_CHECKED=1)")
    x, dy, w, off = make([100], 528, 2048, 3) if kernel == PART else make([150, 0, 290], 512, 384, 3)
    clean = both(x, dy, w, off)
    torch.cuda.synchronize()
    assert F.fp8z1_ffn_timeouts() == 0
    F.fp8z1_checked_ffn_stall(kernel)
    try:
        got = both(x, dy, w, off)
        torch.cuda.synchronize()
    finally:
        F.fp8z1_checked_ffn_stall(0)
    assert F.fp8z1_ffn_timeouts() > 0
    for a, b, hit in zip(got, clean, reached):
        assert bool(a.isnan().any()) == hit
        assert (a.isnan() | (a == b)).all(), "an incomplete number that is not NaN"
    # the next pass is whole
    assert all(torch.equal(a, b) for a, b in zip(both(x, dy, w, off), clean))
    assert F.fp8z1_ffn_timeouts() == 0
