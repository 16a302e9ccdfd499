"""The product's kernel of few rows on more tiles of rows than the rule gives it, which the checked library can be told to."""
import os
import subprocess
import sys

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import build as fp8build
from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests import _ops as R
from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_linear import check

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ALL_FEW = 16
BF16, F32 = torch.bfloat16, torch.float32


def test_on_the_checked_build(lib):
    if F.CHECKED:
        pytest.skip("runs the checked build from the release one")
    fp8build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k", "tiles",
           "tests/test_gpu_ops_linear_few_large.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, FP8Z1_CHECKED="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout and " skipped" not in r.stdout


@pytest.fixture
def all_few(lib):
    if not F.CHECKED:
        pytest.skip("needs the checked build (FP8Z1_CHECKED=1)")
    F.fp8z1_checked_linear_stall(ALL_FEW)
    yield
    F.fp8z1_checked_linear_stall(0)
    assert F.fp8z1_linear_timeouts() == 0


# BF16 rows in pairs and 8-bit rows; 65537 tiles of rows, offsets of x past 2^31
@pytest.mark.parametrize("fp8", [False, True])
def test_more_tiles_than_65535(all_few, fp8):
    tokens, rows, cols = 65536 * 128 + 77, 272, 16
    g = M.gen(6)
    codes, scale = R.fp8_weight(g, rows, cols)
    x = torch.randn((tokens, rows), generator=g, device="cuda", dtype=BF16)
    xs = None
    if fp8:
        x = x.clamp_(-4, 4).to(torch.float8_e4m3fn)
        xs = torch.rand((tokens, 3), generator=g, device="cuda") + 0.5
    y = ops.linear(x, codes, scale, x_scale=xs)
    w = R.decode(codes, scale)
    for i in (0, 65535 * 128, 2**31 // 384, 2**31 // rows, tokens - 300):
        at = slice(max(i - 200, 0), i + 300)
        v = x[at].double()
        if fp8:
            v = v * xs[at].double().repeat_interleave(128, 1)[:, :rows]
        check(y[at], v @ w, v.abs() @ w.abs(), BF16)


@pytest.mark.parametrize("tokens,rows,cols,transposed", [(300, 500, 384, False), (1100, 384, 656, False), (700, 333, 272, True)])
def test_tiles_of_wider_results(all_few, tokens, rows, cols, transposed):
    """Columns' tiles and splits beside several tiles of rows, as the other kernel's."""
    g = M.gen(tokens)
    codes, scale = R.fp8_weight(g, rows, cols)
    inner, outer = (cols, rows) if transposed else (rows, cols)
    x = torch.randn(tokens, inner, generator=g, device="cuda").to(BF16)
    b, r = torch.randn(outer, generator=g, device="cuda"), torch.randn(tokens, outer, generator=g, device="cuda").to(BF16)
    y = ops.linear(x, codes, scale, bias=b, residual=r, transposed=transposed, dtype=F32)
    w = R.decode(codes, scale)
    w = w.T if transposed else w
    want = x.double() @ w + b.double() + r.double()
    check(y, want, x.double().abs() @ w.abs() + b.double().abs() + r.double().abs(), F32)
