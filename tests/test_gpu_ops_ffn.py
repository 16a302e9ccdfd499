"""The gated feed-forward block, forward and backward, against its definition in 64 bits."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

# Weight gradients are FP32 sums of FP32 products.  With sums over up to 2^14 terms, whose roundings (2^-24 each)
# add up like a random walk, in at most three products in a row: 2^-24 * 2^7 * 1.3 = 1e-5 of the norm.
GRAD_TOL = 1e-5


@pytest.fixture(autouse=True)
def _no_timeouts():
    """No wait inside the kernels ran out."""
    yield
    assert F.fp8z1_ffn_timeouts() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make(counts, hidden, inner, seed, rest=0):
    g = gen(seed)
    e = len(counts)
    tokens = sum(counts) + rest
    gu, gus = R.fp8_weight(g, e, hidden, 2 * inner, sigma=1.5 * hidden**-0.5)
    dn, dns = R.fp8_weight(g, e, inner, hidden, sigma=inner**-0.5)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    dy = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    off = torch.tensor([sum(counts[:i]) for i in range(e + 1)], dtype=torch.int32, device="cuda")
    return x, dy, (gu, gus, dn, dns), off


def rel(a, b):
    n = float(b.norm())
    return float((a.double() - b).norm()) / n if n else float(a.double().norm())


def check(x, dy, w, off, got, spans=None, grad_tol=GRAD_TOL):
    y, dx, d_gu, d_dn = got
    want = R.ffn(x, R.decode(w[0], w[1]), R.decode(w[2], w[3]), spans or R.runs(off, w[0].shape[0], x.shape[0]), dy)
    # y: h rounded to 8 bits before the second product, the result once (BF16 has 8 significant bits: 2^-8 each); dx the same with [dg | du];
    # FP32 sums beside that
    for out, k in ((y, "y"), (dx, "dx")):
        if out is not None:
            tol = 1.02 * 2.0**-8 * (want[k].abs() + want[k + "_mag"]) + 1e-30
            assert ((out.double() - want[k]).abs() <= tol).all(), f"{k}: {rel(out, want[k])}"
            # roundings of either sign: about 2^-9.3 of the norm (uniform errors) for each of the two
            assert rel(out, want[k]) <= 2.0**-8
    if d_gu is not None:
        assert rel(d_gu, want["d_gate_up"]) <= grad_tol
        assert rel(d_dn, want["d_down"]) <= grad_tol
        for e, (lo, hi) in enumerate(R.runs(off, w[0].shape[0], x.shape[0]) if spans is None else spans):
            if hi == lo:
                assert not d_gu[e].any() and not d_dn[e].any()


def both(x, dy, w, off):
    y, saved = ops.ffn_forward(x, *w, offsets=off, save=True)
    dx, d_gu, d_dn = ops.ffn_backward(dy, x, saved, *w, offsets=off)
    return y, dx, d_gu, d_dn


@pytest.mark.parametrize("counts,hidden,inner", [
    ([1], 16, 128), ([7], 48, 128), ([129], 304, 256), ([128], 256, 128), ([127], 128, 384), ([257], 1008, 384),
    ([3, 0, 1, 5], 304, 256), ([0, 130, 0], 512, 128), ([1, 128, 129, 255, 256, 2], 256, 256), ([64, 65], 2064, 640),
    ([1100], 640, 256), ([400, 1, 0, 900], 384, 512), ([5] * 40, 128, 128),
])
def test_forward_and_backward(counts, hidden, inner):
    x, dy, w, off = make(counts, hidden, inner, sum(counts) + hidden)
    got = both(x, dy, w, off)
    check(x, dy, w, off, got)
    assert torch.equal(ops.ffn_forward(x, *w, offsets=off), got[0]), "y depends on save"
    again = both(x, dy, w, off)
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "results do not repeat bit for bit"


@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 33, 63])
@pytest.mark.parametrize("experts", [1, 6])
def test_few_tokens(tokens, experts):
    """Serving: single tokens and small batches, dense and spread over experts."""
    counts = [tokens // experts + (i < tokens % experts) for i in range(experts)]
    x, dy, w, off = make(counts, 1040, 384, tokens * 10 + experts)
    y = ops.ffn_forward(x, *w, offsets=off)
    check(x, dy, w, off, (y, None, None, None))
    if experts == 1:
        assert torch.equal(ops.ffn_forward(x, *w), y)


@pytest.mark.parametrize("counts,hidden,inner", [
    ([0, 2, 0, 1], 528, 256), ([0] * 900 + [3, 0, 1], 64, 128), ([0] * 31 + [1], 144, 128), ([9, 0, 0, 5, 1] + [0] * 15 + [2] * 12, 528, 256),
    ([1] * 64, 64, 128), ([4], 7168, 2048), ([3], 16, 128), ([2], 2064, 1152), ([100], 528, 2048), ([60, 0, 3], 2064, 4096),
])
def test_few_tokens_spread_unevenly(counts, hidden, inner):
    """A few tokens on some of many experts, with rows of no expert; products split along inner."""
    x, dy, w, off = make(counts, hidden, inner, 5, rest=1 if len(counts) > 1 else 0)
    n = sum(counts)
    y = ops.ffn_forward(x, *w, offsets=off)
    assert not y[n:].any()
    check(x[:n], dy[:n], w, off, (y[:n], None, None, None))
    assert torch.equal(y, ops.ffn_forward(x, *w, offsets=off))
    assert torch.equal(y, ops.ffn_forward(x, *w, offsets=off, save=True)[0]), "y depends on save"


def test_full_widths_of_the_expert_workload():
    """hidden 7168, inner 2048: three experts of the MoE configuration's widths."""
    x, dy, w, off = make([150, 0, 75], 7168, 2048, 4)
    check(x, dy, w, off, both(x, dy, w, off))


def test_long_run_of_tokens():
    """A weight gradient that sums over thousands of tokens keeps FP32 accuracy."""
    x, dy, w, off = make([5001], 256, 128, 9)
    check(x, dy, w, off, both(x, dy, w, off))


def test_rows_of_no_expert_and_offsets_out_of_range():
    x, dy, w, off = make([70, 30], 256, 128, 1, rest=55)
    y, dx, d_gu, d_dn = both(x, dy, w, off)
    check(x[:100], dy[:100], w, off, (y[:100], dx[:100], d_gu, d_dn))
    assert not y[100:].any() and not dx[100:].any()
    # NaN in rows of no expert reaches nothing
    x2, dy2 = x.clone(), dy.clone()
    x2[100:], dy2[100:] = float("nan"), float("inf")
    assert all(torch.equal(a, b) for a, b in zip(both(x2, dy2, w, off), (y, dx, d_gu, d_dn)))
    # runs that point outside the rows are cut to them
    wild = torch.tensor([0, 70, 1 << 30], dtype=torch.int32, device="cuda")
    got = both(x, dy, w, wild)
    check(x, dy, w, wild, got, spans=[(0, 70), (70, 155)])


def test_strided_rows():
    x, dy, w, off = make([40, 33], 256, 256, 2)
    want = both(x, dy, w, off)
    wide = torch.zeros(73, 3 * 256 + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:264], wide[:, 264:520] = x, dy
    xs, dys = wide[:, 8:264], wide[:, 264:520]
    y, saved = ops.ffn_forward(xs, *w, offsets=off, save=True, out=wide[:, 520:])
    got = (y,) + ops.ffn_backward(dys, xs, saved, *w, offsets=off)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (wide[:, :8] == 0).all()


def test_not_finite_rows_stay_in_their_rows_and_experts():
    for bad in (float("nan"), float("inf"), -float("inf")):
        x, dy, w, off = make([60, 90, 20], 304, 256, 3)
        clean = both(x, dy, w, off)
        x[75, 17] = bad   # a row of expert 1
        y, dx, d_gu, d_dn = both(x, dy, w, off)
        other = [i for i in range(170) if i != 75]
        assert torch.equal(y[other], clean[0][other]) and torch.equal(dx[other], clean[1][other])
        assert not y[75].isfinite().any()
        for e in (0, 2):
            assert torch.equal(d_gu[e], clean[2][e]) and torch.equal(d_dn[e], clean[3][e])
        assert not d_gu[1].isfinite().all() and not d_dn[1].isfinite().all()


def test_not_finite_row_of_a_few_tokens():
    for bad in (float("nan"), float("inf"), -float("inf")):
        x, dy, w, off = make([2, 0, 1], 304, 256, 3)
        clean = ops.ffn_forward(x, *w, offsets=off)
        x[1, 17] = bad
        y = ops.ffn_forward(x, *w, offsets=off)
        assert torch.equal(y[[0, 2]], clean[[0, 2]]) and not y[1].isfinite().any()


def test_uneven_magnitudes():
    """Rows, columns and weight blocks of very different size: every row keeps its own accuracy, and the
    weight gradient that of its sums."""
    x, dy, w, off = make([90, 200], 640, 256, 6)
    x *= torch.logspace(-6, 3, 290, device="cuda")[torch.randperm(290, device="cuda")][:, None].bfloat16()
    dy *= torch.logspace(-3, 5, 290, device="cuda")[torch.randperm(290, device="cuda")][:, None].bfloat16()
    x[:, 5] *= 300   # an outlier channel
    got = both(x, dy, w, off)
    y, dx, d_gu, d_dn = got
    want = R.ffn(x, R.decode(w[0], w[1]), R.decode(w[2], w[3]), R.runs(off, 2, 290), dy)
    for out, k in ((y, "y"), (dx, "dx")):
        err = (out.double() - want[k]).norm(dim=1) / want[k].norm(dim=1)
        assert (err <= 2.0**-8).all()
    assert rel(d_gu, want["d_gate_up"]) <= GRAD_TOL and rel(d_dn, want["d_down"]) <= GRAD_TOL


def test_zero_weights_and_zero_rows():
    x, dy, w, off = make([50, 20], 256, 128, 8)
    w[0][0], w[2][1] = 0, 0x80  # -0 codes
    x[60:] = 0
    got = both(x, dy, w, off)
    check(x, dy, w, off, got)
    assert not got[0].any() and not got[1][:50].any()


def test_gradient_against_differences():
    """Differences of the 64-bit block along random directions in x and both weights."""
    x, dy, w, off = make([9, 30, 0], 160, 128, 12)
    _, dx, d_gu, d_dn = both(x, dy, w, off)
    wgu, wd, spans = R.decode(w[0], w[1]), R.decode(w[2], w[3]), R.runs(off, 3, 39)
    g = gen(1)
    for which in range(3):
        base = [x.double(), wgu, wd]
        v = torch.randn(base[which].shape, generator=g, device="cuda", dtype=torch.float64) * base[which].std()

        def f(step):
            at = list(base)
            at[which] = at[which] + step * v
            return (R.ffn(at[0], at[1], at[2], spans)["y"] * dy.double()).sum()

        eps = 1e-5
        num = float((f(eps) - f(-eps)) / (2 * eps))
        grad = (dx, d_gu, d_dn)[which].double()
        got = float((grad * v).sum())
        # dx's roundings (2^-8 of its norm, in random directions), the weight gradients' 1e-5; eps^2 beside them
        tol = (2.0**-8 if which == 0 else 1e-4) * float(grad.norm()) * float(v.std()) * 4
        assert abs(num - got) <= tol, (which, num, got)


def test_without_dx_and_given_outputs():
    x, dy, w, off = make([33, 40], 256, 128, 21)
    want = both(x, dy, w, off)
    _, saved = ops.ffn_forward(x, *w, offsets=off, save=True)
    a = torch.full(w[0].shape, 7.0, device="cuda")
    b = torch.full(w[2].shape, 7.0, device="cuda")
    dx, d_gu, d_dn = ops.ffn_backward(dy, x, saved, *w, offsets=off, need_dx=False, d_gate_up=a, d_down=b)
    assert dx is None and d_gu is a and d_dn is b
    assert torch.equal(a, want[2]) and torch.equal(b, want[3])


def test_no_tokens():
    x, dy, w, off = make([0, 0], 256, 128, 22)
    y, saved = ops.ffn_forward(x, *w, offsets=off, save=True)
    dx, d_gu, d_dn = ops.ffn_backward(dy, x, saved, *w, offsets=off)
    assert y.shape == (0, 256) and dx.shape == (0, 256) and not d_gu.any() and not d_dn.any()


def test_on_another_stream_and_in_a_graph():
    x, dy, w, off = make([50, 20], 256, 128, 30)
    want = both(x, dy, w, off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        late = x * 1
    y, saved = ops.ffn_forward(late, *w, offsets=off, save=True, stream=s)
    got = (y,) + ops.ffn_backward(dy, late, saved, *w, offsets=off, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # captured once, replayed on new tokens and other runs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(x, dy, w, off)
    x2, dy2, w2, off2 = make([11, 59], 256, 128, 31)
    x.copy_(x2), dy.copy_(dy2), off.copy_(off2)
    for a, b in zip(w, w2):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    want = both(x2, dy2, w2, off2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
