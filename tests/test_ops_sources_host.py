"""What the kernels' sources hold: no GPU."""
import glob
import os
import re

from blockwise_fp8_zero_fold_gb300 import build as fp8build


def test_no_load_writes_to_several_ctas():
    """The library is the data-parallel optimizer's, and every rank of a job loads it: bulk copies that write to several
    CTAs of a cluster at once are for programs of one GPU alone."""
    sources = glob.glob(os.path.join(fp8build.CSRC, "*"))
    assert len(sources) > 15
    for path in sources:
        text = open(path).read()
        # the asm strings of one statement, joined
        text = re.sub(r'"\s*"', "", text)
        for line in re.findall(r"cp\.async\.bulk[^\"]*", text):
            assert "multicast" not in line, f"{os.path.basename(path)}: {line}"
