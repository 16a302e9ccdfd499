"""The 8-bit norm's second result: what does not fit is refused, and what fits reaches the library.  No GPU."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops


@pytest.fixture
def calls(monkeypatch):
    got = []
    monkeypatch.setattr(ops, "_begin", lambda dev, stream: (1, None))
    monkeypatch.setattr(ops, "_scratch", lambda shape, dtype, dev, other: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(F, "fp8z1_rms_norm", lambda *a: got.append(a))
    return got


@pytest.mark.parametrize("out", [lambda x: x.float(), lambda x: x[:3], lambda x: x.t(), lambda x: x[:, :32], lambda x: x[:1].expand(4, 64)])
def test_refused(calls, out):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError):
        ops.rms_norm_fp8(x, w, out=out(x))
    assert not calls


def test_reaches_the_library(calls):
    x, w, wide = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64), torch.zeros(4, 72, dtype=torch.bfloat16)
    out = wide[:, :64]
    codes, scale = ops.rms_norm_fp8(x, w, out=out)
    (a,) = calls
    assert a[11] is out and a[12] == 72 and a[13] is codes and a[14] is scale and codes.dtype == torch.float8_e4m3fn
