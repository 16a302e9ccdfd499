"""The test hook of the feed-forward kernels' waits belongs to the checked build: no GPU."""
from blockwise_fp8_zero_fold_gb300 import build as fp8build
from blockwise_fp8_zero_fold_gb300 import fp8z1 as F


def test_a_release_build_has_no_hook():
    fp8build.build()
    assert F.lib().fp8z1_checked_ffn_stall(1) == F.EINVAL
