"""Calls whose first kernel may start while the one before it ends, captured behind what is not a kernel or is several."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


def state():
    g = M.gen(3)
    codes, scale = R.fp8_weight(g, 256, 20480)
    small, sscale = R.fp8_weight(g, 256, 384)
    x = torch.randn(700, 256, generator=g, device="cuda").bfloat16()
    dy = torch.randn(700, 384, generator=g, device="cuda").bfloat16()
    w = torch.rand(256, generator=g, device="cuda") + 0.5
    q, s = ops.rms_norm_fp8(x, w)
    return codes, scale, small, sscale, x, dy, w, q, s


def calls(st):
    codes, scale, small, sscale, x, dy, w, q, s = st
    return {
        "8-bit rows": lambda: (ops.linear(q, codes, scale, x_scale=s),),
        "few 8-bit rows": lambda: (ops.linear(q[:5], codes, scale, x_scale=s[:5]),),
        "rows": lambda: (ops.linear(x, codes, scale), ops.linear(x[:20], codes, scale)),
        "weight's gradient": lambda: ops.linear_grad(dy, x, small, sscale, need_dx=False)[1:2],
        "weight's gradient of odd rows": lambda: ops.linear_grad(M.strided(dy, 1), x, small, sscale, need_dx=False)[1:2],
        "gradients": lambda: ops.linear_grad(dy, x, small, sscale, bias=True),
        "norm's gradient": lambda: ops.rms_norm_grad(x, x, w),
    }


NAMES = list(calls([None] * 9))
BEFORE = ["nothing", "copy", "memset", "two streams", "itself"]


@pytest.mark.parametrize("before", BEFORE)
@pytest.mark.parametrize("name", NAMES)
def test_captured_behind(name, before):
    st = state()
    call = calls(st)[name]
    want = call()
    x, dy, q, s = st[4], st[5], st[7], st[8]
    kept = [t.clone() for t in (x, dy, q.view(torch.uint8), s)]
    inputs = [x, dy, q.view(torch.uint8), s]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    scratch = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        if before == "copy":  # the inputs arrive in the graph
            for a, b in zip(inputs, kept):
                a.copy_(b)
        elif before == "memset":
            scratch.zero_()
        elif before == "two streams":
            other.wait_stream(side)
            with torch.cuda.stream(other):
                for a, b in list(zip(inputs, kept))[:2]:
                    a.copy_(b)
            for a, b in list(zip(inputs, kept))[2:]:
                a.copy_(b)
            side.wait_stream(other)
        elif before == "itself":
            call()
        got = call()
    for _ in range(20):
        if before in ("copy", "two streams"):
            for a in inputs:
                a.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert F.fp8z1_linear_timeouts() == 0 and F.fp8z1_rms_norm_timeouts() == 0


@pytest.mark.parametrize("name", NAMES)
def test_behind_a_wait_for_another_stream(name):
    """The inputs come from another stream, whose event the call's stream waits for."""
    st = state()
    call = calls(st)[name]
    want = call()
    inputs = [st[4], st[5], st[7].view(torch.uint8), st[8]]
    kept = [t.clone() for t in inputs]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for a in inputs:
            a.zero_()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            torch.cuda._sleep(2_000_000)
            for a, b in zip(inputs, kept):
                a.copy_(b)
        torch.cuda.current_stream().wait_stream(other)
        got = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
