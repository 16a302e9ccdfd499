"""Waits of the norm's gradient that run out: the rows and the weight's gradient that they belong to are NaN, the rest is
whole, and the device goes on.  The checked library leaves a row uncopied, or its place taken; its waits give up after 0.2 s."""
import os
import subprocess
import sys

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import build as fp8build
from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests._gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NEVER_COPIED, NOT_GIVEN_BACK = 1, 2


def test_on_the_checked_build(lib):
    if F.CHECKED:
        pytest.skip("runs the checked build from the release one")
    fp8build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k", "nan",
           "tests/test_gpu_ops_norm_waits.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, FP8Z1_CHECKED="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout and " skipped" not in r.stdout


# two groups of a CTA, 15 warps and 19, and one; of single elements one and two
@pytest.mark.parametrize("dim,dtype", [(7168, torch.bfloat16), (4096, torch.float32), (7168, torch.float32),
                                       (7169, torch.float32), (4097, torch.bfloat16)])
@pytest.mark.parametrize("more", [False, True])
@pytest.mark.parametrize("stall", [NEVER_COPIED, NOT_GIVEN_BACK])
def test_what_a_wait_belongs_to_is_nan(lib, stall, more, dim, dtype):
    if not F.CHECKED:
        pytest.skip("needs the checked build (FP8Z1_CHECKED=1)")
    ctas, g = 152, M.gen(dim)
    rows = ctas * 20 + 5  # more of a CTA than places
    x, dy, dt = (torch.randn(rows, dim, generator=g, device="cuda").to(dtype) for _ in range(3))
    w = torch.rand(dim, generator=g, device="cuda") + 0.5

    def run():
        return ops.rms_norm_grad(dy, x, w, d_total=dt if more else None)

    dx, dw = run()
    torch.cuda.synchronize()
    assert F.fp8z1_rms_norm_timeouts() == 0
    F.fp8z1_checked_rms_norm_stall(stall)
    try:
        got, got_w = run()
        torch.cuda.synchronize()
    finally:
        F.fp8z1_checked_rms_norm_stall(0)
    assert F.fp8z1_rms_norm_timeouts() > 0
    lost = got.isnan().any(1)
    assert (got.isnan().all(1) == lost).all() and torch.equal(got[~lost], dx[~lost]), "an incomplete row that is not NaN"
    # the first CTA's alone, from its first row on, or from the one on that takes the first one's place (16 at most)
    of_first = torch.arange(rows, device="cuda") % ctas == 0
    assert not lost[~of_first].any() and bool(lost[0]) == (stall == NEVER_COPIED) and lost[of_first][16:].all()
    assert got_w.isnan().all()
    # the next pass is whole
    again = run()
    torch.cuda.synchronize()
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and F.fp8z1_rms_norm_timeouts() == 0


# 7, 5, 5, 3, 3 groups, which the 16 places, or the 8 that there would be room for, do not go round evenly
@pytest.mark.parametrize("dim,dtype", [(2048, torch.bfloat16), (3064, torch.bfloat16), (1025, torch.float32), (2049, torch.float32),
                                       (4096, torch.bfloat16)])
@pytest.mark.parametrize("more", [False, True])
def test_a_place_is_one_groups_own_nan(lib, more, dim, dtype):
    """A group does not take a row for its own in a place whose copy, another group's, has not come."""
    test_what_a_wait_belongs_to_is_nan(lib, NEVER_COPIED, more, dim, dtype)
