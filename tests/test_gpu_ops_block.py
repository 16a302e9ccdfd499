"""Norm, routing and matrix products around the feed-forward block, as the example uses them together: a step's gradients,
captured passes, calls on another stream, waits that run out."""
import os
import subprocess
import sys

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import build as fp8build
from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from examples import train_block as X
from tests import _more as M
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_gradients_of_the_whole_step():
    """Against autograd in 64 bits through the decoded weights, the experts as the student chose them.  Beside FP32 the step
    rounds x, h, the experts' h, y, out, last and d_last, d_out, d_y, [dg | du], d_rows, d_h, d_x to BF16's 8 bits, 2^-9 of the
    norm at most each (uniform errors: half that), and their effects add up over the chain: 13 * 2^-9 = 2.5 %.  The router's and
    norms' gradients are sums of what nearly cancels (a softmax's, a norm's: the part along the row is taken out): twice that."""
    s = X.Student(vocab=503, hidden=144, inner=128, experts=16)
    s.norms.add_(torch.randn(2, 144, generator=M.gen(4), device="cuda") * 0.2)
    ids = torch.randint(s.vocab, (301,), generator=M.gen(3), device="cuda")
    t_ids, t_logits = X.teacher(s.vocab, 9)
    scale = s.opt.scaler.scale
    _, (_, _, chosen, _, _, _, _, _) = s.forward(ids, save=True)
    loss = s.gradients(ids, t_ids[ids], t_logits[ids]).mean()

    w = [R.decode(c, v).requires_grad_() for c, v in zip(s.codes, s.scales)]
    norms = s.norms.double().requires_grad_()
    norm = lambda x, k: x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * norms[k]  # noqa: E731
    x = s.alpha * w[0][0][ids]
    h = norm(x, 0)
    p = (h @ w[1][0]).gather(1, chosen).softmax(1)
    each = torch.einsum("th,ehf->tef", h, w[2])
    gate, up = each.chunk(2, 2)
    y = torch.einsum("tef,efh->teh", torch.nn.functional.silu(gate) * up, w[3])
    out = x + (p[:, :, None] * y.gather(1, chosen[:, :, None].expand(-1, -1, 144))).sum(1)
    q = (norm(out, 1) @ w[0][0].T).log_softmax(1)
    t = t_logits[ids].double().log_softmax(1)
    want = (t.exp() * (t - q.gather(1, t_ids[ids].long()))).sum(1).mean()
    want.backward()
    step = 13 * 2.0**-9
    assert abs(float(loss) - want.item()) <= step * abs(want.item())
    for got, ref, n in zip(s.grads + [s.norms.grad], w + [norms], (1, 2, 1, 1, 2)):
        ref = ref.grad * scale
        assert float((got.double() - ref).norm()) <= n * step * float(ref.norm())


def test_the_example_runs():
    losses = X.main(steps=3, tokens=700)
    assert len(losses) == 3 and all(v == v and v < float("inf") for v in losses)


def test_serving_in_8_bits():
    """Logits by way of 8-bit rows against those of BF16 rows: a row's 256 numbers are off by 2^-4 of themselves at most each, of
    either sign, 2^-5.3 of the norm for uniform errors beside 2^-9 of BF16's; a logit by as much of its terms' root sum of squares,
    at most five times that in any of 500 x 1000."""
    s = X.Student()
    ids = torch.randint(s.vocab, (500,), generator=M.gen(1), device="cuda")
    z = s.logits(ids)
    last = ops.rms_norm(s.forward(ids), s.norms[1])
    table = R.decode(s.codes[0], s.scales[0])[0]
    want = last.double() @ table.T
    rms = (last.double().square() @ table.square().T).sqrt()
    assert ((z.double() - want).abs() <= 5 * 2.0**-4.9 * rms).all()
    # a token by itself takes other kernels
    assert ((s.logits(ids[:1]).double() - want[:1]).abs() <= 5 * 2.0**-4.9 * rms[:1]).all()


def calls():
    """Each operator, forward and backward, few rows and many."""
    g = M.gen(5)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, res, dy, wn = n(700, 256), n(700, 256), n(700, 256), torch.rand(256, generator=g, device="cuda") + 0.5
    wide, dwide, wwide = n(700, 2056), n(700, 2056), torch.rand(2056, generator=g, device="cuda") + 0.5
    ids = torch.randint(-1, 9, (700, 3), generator=g, device="cuda", dtype=torch.int32)
    cw = torch.rand(700, 3, generator=g, device="cuda")
    rows, d_rows = n(2100, 256), n(2100, 256)
    codes, scale = R.fp8_weight(g, 256, 384)
    bias = torch.randn(384, generator=g, device="cuda")
    dz = n(700, 384)
    big, bscale = R.fp8_weight(g, 256, 20480)

    def route(stream):
        r = ops.route(ids, 9, stream=stream)
        return (r.offsets, r.place, ops.dispatch(x, r, stream=stream), ops.combine(rows, r, cw, residual=res, stream=stream),
                ops.dispatch_grad(d_rows, r, stream=stream), *ops.combine_grad(dy, rows, r, cw, stream=stream))

    def linear(stream):
        y, pre = ops.linear(x, codes, scale, bias=bias, activation="silu", save=True, stream=stream)
        few = ops.linear(x[:9], codes, scale, stream=stream)
        many = ops.linear(x, big, bscale, stream=stream)
        q, s = ops.rms_norm_fp8(x, wn, stream=stream)
        return (y, pre, few, many, ops.linear(q, codes, scale, x_scale=s, stream=stream),
                *ops.linear_grad(dz, x, codes, scale, activation="silu", pre=pre, bias=True, stream=stream),
                *ops.linear_grad(dz, x, codes, scale, bias=True, stream=stream))

    return {
        "norm": lambda stream: (*ops.rms_norm(x, wn, residual=res, stream=stream), *ops.rms_norm_fp8(x, wn, residual=res, stream=stream),
                                *ops.rms_norm_grad(dy, x, wn, stream=stream),
                                *ops.rms_norm_grad(dwide, wide, wwide, d_total=dwide, stream=stream)),
        "route": route,
        "linear": linear,
    }


LONG = 20_000_000  # clocks: about 10 ms, far longer than the calls


@pytest.mark.parametrize("name", ["norm", "route", "linear"])
def test_beside_the_same_call_on_the_current_stream(name):
    """The current stream's call waits behind a long kernel while its freed workspace lies in the pool."""
    call = calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(LONG)
    first = call(None)
    second = call(s)
    third = call(None)
    torch.cuda.synchronize()
    for got in (first, second, third):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["norm", "route", "linear"])
def test_beside_a_read_of_memory_that_is_freed(name):
    """Blocks of the sizes that the call allocates, still to be read by the current stream, are not written."""
    call = calls()[name]
    sizes = [t.numel() * t.element_size() for t in call(None)] + [1 << k for k in range(12, 25)]
    s = torch.cuda.Stream()
    call(s)
    torch.cuda.synchronize()
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    kept = [torch.empty_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    for k, b in zip(kept, blocks):
        k.copy_(b)
    del blocks, b
    call(s)
    torch.cuda.synchronize()
    assert all((k == 7).all() for k in kept)


@pytest.mark.parametrize("name", ["norm", "route", "linear"])
def test_a_pass_can_be_captured(name):
    """In two CUDA graphs, replayed in turn, beside eager calls; a third of other inputs in their places."""
    call = calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(None)
    torch.cuda.current_stream().wait_stream(side)
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            got.append(call(None))
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        eager = call(None)
    torch.cuda.synchronize()
    for outs in got + [eager]:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_a_captured_pass_reads_its_inputs_anew():
    s = X.Student()
    ids = torch.randint(s.vocab, (600,), generator=M.gen(6), device="cuda")
    other = torch.randint(s.vocab, (600,), generator=M.gen(7), device="cuda")
    want = s.forward(other), s.logits(other)
    x = ids.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.forward(x), s.logits(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.forward(x), s.logits(x)
    x.copy_(other)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_products_while_other_kernels_hold_the_sms():
    """Clusters that split K start when they can: no CTA reads another's sums before they are there."""
    g = M.gen(8)
    codes, scale = R.fp8_weight(g, 4096, 256)
    x = torch.randn(5, 4096, generator=g, device="cuda").bfloat16()
    big = torch.randn(300, 4096, generator=g, device="cuda").bfloat16()
    want, want_big = ops.linear(x, codes, scale), ops.linear(big, codes, scale)
    a = torch.randn(2048, 2048, generator=g, device="cuda").bfloat16()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(100):
        with torch.cuda.stream(s):
            a @ a
        got.append((ops.linear(x, codes, scale), ops.linear(big, codes, scale)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want_big) for a, b in got)
    assert F.fp8z1_linear_timeouts() == 0


# ---- waits that run out: what they belong to is NaN, the rest is whole, and the device goes on ----------------------


def test_waits_on_the_checked_build(lib):  # noqa: F811
    if F.CHECKED:
        pytest.skip("runs the checked build from the release one")
    fp8build.build(checked=True)
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_gpu_ops_block.py::test_what_a_wait_belongs_to_is_nan"]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, FP8Z1_CHECKED="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout and " skipped" not in r.stdout


MANY, FEW, D_WEIGHT, D_TURNED = (1 << i for i in range(4))


# which of the outputs (y of many rows, y of few, dx, d_weight, d_weight of a transposed weight) a kernel's sums reach
@pytest.mark.parametrize("kernel,reached", [
    (MANY, (True, False, False, False, False)), (FEW, (False, True, True, False, False)), (D_WEIGHT, (False, False, False, True, False)),
    (D_TURNED, (False, False, False, False, True))])
def test_what_a_wait_belongs_to_is_nan(lib, kernel, reached):  # noqa: F811
    if not F.CHECKED:
        pytest.skip("needs the checked build (FP8Z1_CHECKED=1)")
    g = M.gen(9)
    codes, scale = R.fp8_weight(g, 384, 20480)
    x = torch.randn(600, 384, generator=g, device="cuda").bfloat16()
    small, sscale = R.fp8_weight(g, 384, 384)
    dy = torch.randn(600, 384, generator=g, device="cuda").bfloat16()

    def run():
        return (ops.linear(x, codes, scale), ops.linear(x[:40], codes, scale),
                *ops.linear_grad(dy, x, small, sscale)[:2], ops.linear_grad(dy, x, small, sscale, transposed=True, need_dx=False)[1])

    clean = run()
    torch.cuda.synchronize()
    assert F.fp8z1_linear_timeouts() == 0
    F.fp8z1_checked_linear_stall(kernel)
    try:
        got = run()
        torch.cuda.synchronize()
    finally:
        F.fp8z1_checked_linear_stall(0)
    assert F.fp8z1_linear_timeouts() > 0
    for a, b, hit in zip(got, clean, reached):
        assert bool(a.isnan().any()) == hit
        assert (a.isnan() | (a == b)).all(), "an incomplete number that is not NaN"
    # the next pass is whole
    assert all(torch.equal(a, b) for a, b in zip(run(), clean))
    assert F.fp8z1_linear_timeouts() == 0
