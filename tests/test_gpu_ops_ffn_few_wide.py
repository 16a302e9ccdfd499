"""Two to four tokens of wide blocks, on either side of where their products change."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from tests._gpu import lib  # noqa: F401
from tests.test_gpu_ops_ffn import check, make

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


@pytest.mark.parametrize("counts,hidden,inner,vectors", [
    ([1], 4096, 14336, True), ([2], 4096, 14336, False), ([4], 4096, 14336, False), ([4], 7168, 2048, True),
    ([2, 0, 2], 4096, 8192, False), ([1, 0, 1], 4096, 5632, True), ([3], 2064, 14336, True)])
def test_two_to_four_tokens_of_wide_blocks(counts, hidden, inner, vectors):
    x, dy, w, off = make(counts, hidden, inner, 6)
    y = ops.ffn_forward(x, *w, offsets=off)
    check(x, dy, w, off, (y, None, None, None))
    before = F.fp8z1_kernel_launches()
    again = ops.ffn_forward(x, *w, offsets=off)
    assert (F.fp8z1_kernel_launches() - before == 2) == vectors  # matrix-vector products: two launches
    assert torch.equal(y, again)
    assert F.fp8z1_ffn_timeouts() == 0
