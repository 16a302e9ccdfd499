"""Results in memory that a call's inputs lie in too, where that is right: in their place, and between their rows."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

BF16, F32 = torch.bfloat16, torch.float32


def beside(*tensors):
    """The same tensors as columns of one buffer."""
    both = torch.cat(tensors, 1)
    return torch.split(both, [t.shape[1] for t in tensors], 1)


def product(tokens, seed):
    g = M.gen(seed)
    codes, scale = R.fp8_weight(g, 256, 256)
    x, r, dy = (torch.randn(tokens, 256, generator=g, device="cuda").bfloat16() for _ in range(3))
    return codes, scale, x, r, dy


@pytest.mark.parametrize("tokens", [1, 30, 700])
def test_product(tokens):
    codes, scale, x, r, _ = product(tokens, tokens)
    want = ops.linear(x, codes, scale, residual=r)
    xs, rs, out = beside(x, r, torch.zeros_like(x))
    assert torch.equal(ops.linear(xs, codes, scale, residual=rs, out=out), want) and torch.equal(xs, x) and torch.equal(rs, r)
    assert torch.equal(ops.linear(xs, codes, scale, residual=rs, out=rs), want) and torch.equal(xs, x)
    # BF16 rows have been read when the first result is written
    assert torch.equal(ops.linear(xs, codes, scale, residual=r, out=xs), want)


@pytest.mark.parametrize("tokens", [1, 30, 700])
@pytest.mark.parametrize("act", [None, "silu"])
def test_products_gradients(tokens, act):
    """dx in dy's place where d_weight is not wanted, or dz is not dy itself."""
    codes, scale, x, r, dy = product(tokens, tokens)
    _, pre = ops.linear(x, codes, scale, activation=act, save=True)
    want = ops.linear_grad(dy, x, codes, scale, activation=act, pre=pre, bias=True)
    d = F.fp8z1_linear_dims(tokens, 256, 256, 0, F.ACT_SILU if act else F.ACT_NONE, F.BF16, F.BF16)
    ws = torch.empty(F.fp8z1_linear_sizes(d)[1], dtype=torch.uint8, device="cuda")
    dx, dw, db = dy.clone(), torch.empty_like(want[1]) if act else None, torch.empty_like(want[2])
    F.fp8z1_linear_grad(d, dx, 256, x, 256, codes, scale, pre, dx, 256, dw, db, ws, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(dx, want[0]) and torch.equal(db, want[2]) and (dw is None or torch.equal(dw, want[1]))


@pytest.mark.parametrize("rows", [1, 5, 900])
@pytest.mark.parametrize("dim", [96, 1536, 2001])
def test_norm(rows, dim):
    g = M.gen(dim)
    x, r, dy, dt = (torch.randn(rows, dim, generator=g, device="cuda").bfloat16() for _ in range(4))
    w = torch.rand(dim, generator=g, device="cuda") + 0.5
    y, total = ops.rms_norm(x, w, residual=r)
    dx, dw = ops.rms_norm_grad(dy, total, w, d_total=dt)
    xs, rs, ys, ts = beside(x, r, torch.zeros_like(x), torch.zeros_like(x))
    got = ops.rms_norm(xs, w, residual=rs, out=ys, total=ts)
    assert torch.equal(got[0], y) and torch.equal(got[1], total) and torch.equal(xs, x) and torch.equal(rs, r)
    got = ops.rms_norm(xs, w, residual=rs, out=rs, total=xs)
    assert torch.equal(got[0], y) and torch.equal(got[1], total)
    for k in range(4):
        dys, ss, dts, more = beside(dy, total, dt, torch.zeros_like(x))
        got = ops.rms_norm_grad(dys, ss, w, d_total=dts, dx=(dys, ss, dts, more)[k])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("dim", [64, 1001])
@pytest.mark.parametrize("tokens", [1, 200])
def test_rows(tokens, dim):
    g = M.gen(dim)
    top, experts = 3, 7
    r = ops.route(torch.randint(-1, experts, (tokens, top), generator=g, device="cuda"), experts)
    x, res, dy = (torch.randn(tokens, dim, generator=g, device="cuda").bfloat16() for _ in range(3))
    rows = torch.randn(tokens * top, dim, generator=g, device="cuda").bfloat16()
    w = torch.rand(tokens, top, generator=g, device="cuda")
    got, y, d = ops.dispatch(x, r), ops.combine(rows, r, w, residual=res), ops.combine_grad(dy, rows, r, w)
    # tokens' rows and the experts' as columns of one buffer
    wide = torch.zeros(tokens * top, 3 * dim, dtype=BF16, device="cuda")
    xs, out, ys = wide[:tokens, :dim], wide[:, dim:2 * dim], wide[:tokens, 2 * dim:]
    xs.copy_(x)
    assert torch.equal(ops.dispatch(xs, r, out=out), got) and torch.equal(xs, x)
    out.copy_(rows)
    xs.copy_(res)
    assert torch.equal(ops.combine(out, r, w, residual=xs, out=ys), y) and torch.equal(out, rows) and torch.equal(xs, res)
    assert torch.equal(ops.combine(out, r, w, residual=xs, out=xs), y) and torch.equal(out, rows)
    xs.copy_(dy)
    again = ops.combine_grad(xs, out, r, w, out=out)  # in the rows' place
    assert torch.equal(again[0], d[0]) and torch.equal(again[1], d[1]) and torch.equal(xs, dy)
    # behind one another in one buffer
    long = torch.zeros(tokens * (top + 1), dim, dtype=BF16, device="cuda")
    long[:tokens] = x
    assert torch.equal(ops.dispatch(long[:tokens], r, out=long[tokens:]), got)
    with pytest.raises(F.Fp8z1Error):
        ops.dispatch(long[:tokens], r, out=long[tokens - 1:-1])
    with pytest.raises(F.Fp8z1Error):
        ops.combine(rows, r, w, out=rows[tokens:2 * tokens])
