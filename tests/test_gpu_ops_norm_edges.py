"""The norm's gradient on both sides of the widths where its threads change: groups of a CTA, 19 warps, a row's own CTA, no ring."""
import pytest
import torch

from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_norm import test_gradient as gradient

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


# 15 warps in groups: 1536, 2560; 19 warps from 3585 to 4608; 32 elements a thread beyond 7680; more than 15 warps beyond 15360
@pytest.mark.parametrize("dim", [1024, 1025, 1032, 1536, 1537, 2559, 2560, 2561, 3583, 3584, 3585, 3592, 4608, 4609, 4616, 7679,
                                 7681, 7688, 15360, 15361, 15368])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_edges(dim, dtype):
    gradient(640 if dim < 8000 else 310, dim, dtype)
