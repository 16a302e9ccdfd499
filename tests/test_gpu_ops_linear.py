"""The matrix product with an FP8 weight and its gradients, against their definition in 64 bits."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

BF16, F32 = torch.bfloat16, torch.float32

# FP32 sums of exact products.  Tensor memory adds 32 at a time and cuts off what lies below the last place of the larger
# number (2^-23 of the magnitudes for each of 4 or, with 256 rows of 16, 16 additions), then at most 2^7 blocks are added in
# registers with 2^-24 each, mostly of either sign: 2^-23 * 16 + 2^-24 * 2^7 / 4 < 2^-17.5 of the terms' magnitudes.
SUMS = 2.0**-17


@pytest.fixture(autouse=True)
def _no_timeouts():
    """No wait inside the kernels ran out."""
    yield
    assert F.fp8z1_linear_timeouts() == 0


def make(tokens, rows, cols, transposed, seed, x="bf16", dy=BF16):
    g = M.gen(seed)
    inner, outer = (cols, rows) if transposed else (rows, cols)
    codes, scale = R.fp8_weight(g, rows, cols, sigma=inner**-0.5)
    w = R.decode(codes[None], scale[None])[0]
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s = dict(codes=codes, scale=scale, w=w.T if transposed else w, x=n(tokens, inner).bfloat16(), x_scale=None,
             bias=n(outer), residual=n(tokens, outer).bfloat16(), dy=n(tokens, outer).to(dy))
    s["xv"] = s["x"].double()
    if x == "fp8":
        s["x"] = (n(tokens, inner) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["x_scale"] = (torch.rand(tokens, -(-inner // 128), generator=g, device="cuda") + 0.5) / 100
        s["xv"] = s["x"].double() * s["x_scale"].double().repeat_interleave(128, 1)[:, :inner]
    return s


def check(got, want, mag, dtype, sums=SUMS):
    err = (got.double() - want).abs()
    tol = M.half_step(dtype) * 1.01 * want.abs() + sums * mag + 1e-37
    assert (err <= tol).all(), f"{float((err / tol).max())} at {int((err / tol).argmax())}"


def forward(s, transposed, act, bias, residual, dtype, save=False, out=None):
    b, r = s["bias"] if bias else None, s["residual"] if residual else None
    got = ops.linear(s["x"], s["codes"], s["scale"], x_scale=s["x_scale"], bias=b, activation=act, residual=r,
                     transposed=transposed, dtype=dtype, save=save, out=out)
    y, pre = got if save else (got, None)
    z, mag = s["xv"] @ s["w"], s["xv"].abs() @ s["w"].abs()
    if bias:
        z, mag = z + b.double(), mag + b.double().abs()
    if save:
        check(pre, z, mag, F32)
    want = M.gate(z, act)[0]
    # an activation's slope is at most 1.13; its own FP32 arithmetic 2^-19 of z
    mag = mag * (1.13 if act else 1.0)
    if residual:
        want, mag = want + r.double(), mag + r.double().abs()
    check(y, want, mag, dtype)
    return y, pre


# few rows (16, 32, 64, 128 a CTA), rows that end inside a tile, many rows; columns and rows that end inside a block
TOKENS = [1, 2, 15, 16, 17, 33, 61, 64, 65, 128, 129, 300, 700]
WEIGHTS = [(16, 16, False), (128, 128, False), (304, 272, False), (1000, 144, False), (7, 32, False), (129, 640, False),
           (16, 16, True), (128, 256, True), (1001, 272, True), (1, 16, True), (131, 1040, True)]


@pytest.mark.parametrize("rows,cols,transposed", WEIGHTS)
@pytest.mark.parametrize("tokens", TOKENS)
def test_product(tokens, rows, cols, transposed):
    s = make(tokens, rows, cols, transposed, tokens + rows)
    forward(s, transposed, None, False, False, BF16)
    forward(s, transposed, "silu", True, True, F32, save=True)


@pytest.mark.parametrize("rows,cols,transposed", [w for w in WEIGHTS if (w[1] if w[2] else w[0]) % 16 == 0])
@pytest.mark.parametrize("tokens", TOKENS)
def test_product_of_8_bit_rows(tokens, rows, cols, transposed):
    s = make(tokens, rows, cols, transposed, tokens + rows, x="fp8")
    forward(s, transposed, None, False, False, F32)
    forward(s, transposed, "gelu_tanh", True, True, BF16, save=True)


@pytest.mark.parametrize("act", [None, "silu", "gelu_tanh"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [5, 100, 1500])
def test_what_joins_the_sums(tokens, dtype, residual, bias, act):
    s = make(tokens, 512, 2064, False, tokens)
    plain = ops.linear(s["x"], s["codes"], s["scale"], bias=s["bias"] if bias else None, activation=act,
                       residual=s["residual"] if residual else None, dtype=dtype)
    y, _ = forward(s, False, act, bias, residual, dtype, save=True)
    assert torch.equal(y, plain)  # y does not depend on `save`, and repeats


@pytest.mark.parametrize("tokens,rows,cols,transposed,x", [
    (1, 4096, 14336, False, "fp8"), (16, 7168, 4096, False, "bf16"), (61, 14336, 4096, True, "bf16"), (128, 4096, 4096, False, "fp8"),
    (2051, 4096, 2048, False, "bf16"), (4100, 1024, 4096, False, "fp8"), (3000, 4097, 512, True, "fp8"), (5000, 640, 7168, True, "bf16")])
def test_larger_products(tokens, rows, cols, transposed, x):
    s = make(tokens, rows, cols, transposed, tokens, x)
    forward(s, transposed, None, False, True, F32)


@pytest.mark.parametrize("x", ["bf16", "fp8"])
@pytest.mark.parametrize("tokens", [257, 300, 320])
def test_rows_beyond_whole_tiles(tokens, x):
    """A few rows past 256 over many columns: those rows' result is the others' kind, in every form."""
    for transposed in (False, True):
        s = make(tokens, *((19712, 256) if transposed else (256, 19712)), transposed, tokens, x)
        for pad, dtype in ((0, BF16), (3, F32)):
            out = M.strided(torch.zeros(tokens, 19712, dtype=dtype, device="cuda"), pad)
            y, pre = forward(s, transposed, "silu", True, True, dtype, save=True, out=out)
            again, pre2 = forward(s, transposed, "silu", True, True, dtype, save=True)
            assert torch.equal(y, again) and torch.equal(pre, pre2)


@pytest.mark.parametrize("tokens", [3, 90, 800])
@pytest.mark.parametrize("pad,at", [(8, 0), (1, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_offsets(tokens, pad, at, dtype):
    s = make(tokens, 264, 144, False, tokens)
    want = forward(s, False, "silu", True, True, dtype)[0]
    s["x"], s["residual"] = M.strided(s["x"], pad, at), M.strided(s["residual"], pad, at)
    out = M.strided(torch.zeros_like(want), pad, at)
    y, _ = forward(s, False, "silu", True, True, dtype, save=True, out=out)
    assert y is out and torch.equal(y, want)
    if pad and tokens > 1:
        assert out.as_strided((tokens - 1, pad), (144 + pad, 1), out.storage_offset() + 144).isnan().all()


@pytest.mark.parametrize("tokens", [4, 200, 600])
def test_8_bit_rows_of_another_stride(tokens):
    s = make(tokens, 160, 128, False, tokens, "fp8")
    want = forward(s, False, None, False, False, BF16)[0]
    wide = torch.zeros(tokens, 192, dtype=torch.uint8, device="cuda")
    wide[:, :160] = s["x"].view(torch.uint8)
    wide[:, 160:] = 127  # NaN behind each row
    s["x"] = wide.view(torch.float8_e4m3fn)[:, :160]
    assert torch.equal(forward(s, False, None, False, False, BF16)[0], want)


@pytest.mark.parametrize("tokens", [1, 40, 500])
def test_result_over_the_residual(tokens):
    s = make(tokens, 256, 384, False, tokens)
    want = ops.linear(s["x"], s["codes"], s["scale"], residual=s["residual"])
    got = ops.linear(s["x"], s["codes"], s["scale"], residual=s["residual"], out=s["residual"])
    assert got is s["residual"] and torch.equal(got, want)


@pytest.mark.parametrize("x", ["bf16", "fp8"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bias,act,residual", [(False, None, False), (True, None, False), (True, "silu", True), (False, "gelu_tanh", False)])
@pytest.mark.parametrize("rows,cols,transposed,pad", [(1024, 4112, False, 0), (1024, 4112, False, 16), (1024, 4112, False, 3),
                                                      (4105, 1024, True, 0), (4105, 1024, True, 1)])
def test_ends_of_large_tiles(rows, cols, transposed, pad, bias, act, residual, dtype, x):
    """Enough rows and columns for the widest tiles, the last ones cut off; results on 16 bytes, and not."""
    s = make(2051, rows, cols, transposed, rows + pad, x)
    outer = rows if transposed else cols
    out = torch.full((2051, outer + pad), 7.0, dtype=dtype, device="cuda")
    forward(s, transposed, act, bias, residual, dtype, save=act is not None, out=out[:, :outer])
    assert (out[:, outer:] == 7.0).all()


def test_other_rows_do_not_matter():
    """An infinity, a NaN, and the largest and smallest numbers leave the other rows' results as they were."""
    for tokens in (6, 300):
        s = make(tokens, 256, 128, False, 3)
        want = forward(s, False, None, False, False, F32)[0]
        s["x"][1, 5], s["x"][2, 7] = float("inf"), float("nan")
        s["x"][3] *= 1e30
        s["x"][4] = 0
        y = ops.linear(s["x"], s["codes"], s["scale"], dtype=F32)
        some = [0, 5] + list(range(6, tokens))
        assert torch.equal(y[some], want[some])
        assert not y[1].isfinite().any() and not y[2].isfinite().any() and not y[4].any()
        check(y[3], s["x"][3].double() @ s["w"], s["x"][3].double().abs() @ s["w"].abs(), F32)


def rel(a, b):
    n = float(b.norm())
    return float((a.double() - b).norm()) / n if n else float(a.double().norm())


def backward(s, transposed, act, dtype, bias=True):
    pre = None
    if act:
        _, pre = ops.linear(s["x"], s["codes"], s["scale"], bias=s["bias"], activation=act, transposed=transposed, save=True)
    kw = dict(activation=act, pre=pre, transposed=transposed, bias=bias)
    dx, dw, db = ops.linear_grad(s["dy"], s["x"], s["codes"], s["scale"], **kw)
    dz = s["dy"].double() * (M.gate(pre.double(), act)[1] if act else 1.0)
    x, w = s["xv"], s["w"]
    # an activation's slope in FP32: 2^-20 of 1.13 or so, of dy
    off = s["dy"].double().abs() * 2.0**-20 if act else torch.zeros_like(dz)
    exact = act is None and dtype == BF16
    mag = dz.abs() @ w.abs().T
    tol = M.half_step(BF16) * 1.01 * (dz @ w.T).abs() + SUMS * mag + off @ w.abs().T + 1e-37
    if not exact:  # dz to 9 bits, or 2^-17 of the largest of its 128 neighbours
        pad = torch.zeros(dz.shape[0], -(-dz.shape[1] // 128) * 128, dtype=torch.float64, device="cuda")
        pad[:, : dz.shape[1]] = dz.abs()
        top = pad.view(dz.shape[0], -1, 128).amax(2).repeat_interleave(128, 1)[:, : dz.shape[1]]
        tol = tol + 2.0**-9 * 1.01 * mag + 2.0**-17 * (top @ w.abs().T)
    err = (dx.double() - dz @ w.T).abs()
    assert (err <= tol).all(), float((err / tol).max())
    want = dz.T @ x if transposed else x.T @ dz
    mag = dz.abs().T @ x.abs() if transposed else x.abs().T @ dz.abs()
    more = off.T @ x.abs() if transposed else x.abs().T @ off
    err = (dw.double() - want).abs()
    assert (err <= SUMS * mag + more + 1e-37).all(), float((err / (SUMS * mag + more)).max())
    assert rel(dw, want) <= 2e-6  # roundings of either sign: 7e-7 of the norm by 256 rows in tensor memory, 2^-22 by the terms
    if bias:
        n = s["dy"].shape[0]
        # 8 rows in a row, 32 warps, then n / 256 blocks in 32 threads and a tree
        assert ((db.double() - dz.sum(0)).abs() <= 2.0**-24 * (48 + n / 2048) * dz.abs().sum(0) + off.sum(0) + 1e-37).all()
    again = ops.linear_grad(s["dy"], s["x"], s["codes"], s["scale"], **kw)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again) if a is not None)
    return dx, dw, db


@pytest.mark.parametrize("rows,cols,transposed", WEIGHTS + [(520, 400, False), (520, 400, True)])
@pytest.mark.parametrize("tokens", [1, 7, 16, 63, 65, 128, 255, 257, 600])
@pytest.mark.parametrize("act,dtype", [(None, BF16), (None, F32), ("silu", BF16), ("gelu_tanh", F32)])
def test_gradients(tokens, rows, cols, transposed, act, dtype):
    s = make(tokens, rows, cols, transposed, tokens + rows, dy=dtype)
    backward(s, transposed, act, dtype)


@pytest.mark.parametrize("tokens,rows,cols,transposed,act,dtype", [
    (2051, 1024, 4096, False, "gelu_tanh", BF16), (8192, 512, 512, False, None, BF16), (3000, 5001, 1024, True, None, F32),
    (1500, 4096, 2064, True, None, BF16), (4099, 2048, 272, False, "silu", F32)])
def test_larger_gradients(tokens, rows, cols, transposed, act, dtype):
    backward(make(tokens, rows, cols, transposed, tokens, dy=dtype), transposed, act, dtype)


@pytest.mark.parametrize("pad,at", [(8, 0), (1, 0), (0, 1), (4, 4)])
@pytest.mark.parametrize("act,dtype", [(None, BF16), (None, F32), ("silu", BF16)])
def test_gradients_of_other_strides(pad, at, act, dtype):
    for tokens in (5, 300):
        s = make(tokens, 200, 144, False, tokens, dy=dtype)
        want = backward(s, False, act, dtype)
        s["x"], s["dy"] = M.strided(s["x"], pad, at), M.strided(s["dy"], pad, at)
        got = backward(s, False, act, dtype)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("act,dtype", [(None, BF16), ("silu", BF16), (None, F32)])
def test_some_of_the_gradients(act, dtype):
    s = make(130, 272, 160, False, 8, dy=dtype)
    pre = ops.linear(s["x"], s["codes"], s["scale"], activation=act, save=True)[1] if act else None
    call = lambda **kw: ops.linear_grad(s["dy"], s["x"], s["codes"], s["scale"], activation=act, pre=pre, **kw)  # noqa: E731
    full = call(bias=True)
    for dx in (False, True):
        for dw in (False, True):
            for db in (False, True):
                if not (dx or dw or db):
                    continue
                got = call(need_dx=dx, need_weight=dw, bias=db)
                for want, a, b in zip((dx, dw, db), got, full):
                    assert (a is None) != want and (a is None or torch.equal(a, b))
    given = torch.full_like(full[1], 7.0), torch.full_like(full[2], 7.0)
    got = call(bias=True, d_weight=given[0], d_bias=given[1])
    assert got[1] is given[0] and got[2] is given[1] and all(torch.equal(a, b) for a, b in zip(got, full))


def test_gradients_against_differences():
    s = make(6, 48, 32, False, 2, dy=F32)
    pre = ops.linear(s["x"], s["codes"], s["scale"], bias=s["bias"], activation="gelu_tanh", save=True, dtype=F32)[1]
    dx, dw, db = ops.linear_grad(s["dy"], s["x"], s["codes"], s["scale"], activation="gelu_tanh", pre=pre, bias=True)

    def f(x, w, b):
        return float((s["dy"].double() * M.gate(x @ w + b, "gelu_tanh")[0]).sum())

    at = [s["xv"], s["w"], s["bias"].double()]
    for k, (got, tol) in enumerate(((dx, 2.0**-7), (dw, 1e-4), (db, 1e-4))):
        for i in (0, got.numel() // 2, got.numel() - 1):
            h = torch.zeros_like(at[k])
            h.reshape(-1)[i] = 1e-5
            up, down = ([a + sign * h if j == k else a for j, a in enumerate(at)] for sign in (1, -1))
            d = (f(*up) - f(*down)) / 2e-5
            assert abs(float(got.reshape(-1)[i]) - d) <= tol * max(1.0, abs(d)) * 2


def test_columns_of_small_numbers_keep_theirs():
    """dz's columns 2^-60 of their neighbours, and rows of x beside an outlier, lose nothing in d_weight."""
    s = make(700, 256, 144, False, 4, dy=F32)
    s["dy"][:, 3] *= 2.0**-60
    s["dy"][:300, 5] *= 2.0**-30
    s["x"][10] *= 2.0**12
    s["xv"] = s["x"].double()
    dw = backward(s, False, None, F32)[1]
    want = s["xv"].T @ s["dy"].double()
    for c in (3, 5):
        assert rel(dw[:, c], want[:, c]) <= 2e-6


def test_infinities_in_the_gradients():
    """An infinity in x or dy touches its row of dx, its row or column of d_weight and its d_bias alone."""
    for act, dtype in ((None, BF16), (None, F32)):
        s = make(300, 256, 144, False, 4, dy=dtype)
        want = ops.linear_grad(s["dy"], s["x"], s["codes"], s["scale"], bias=True)
        s["x"][7, 9] = float("inf")
        s["dy"][20, 30] = float("inf")
        dx, dw, db = ops.linear_grad(s["dy"], s["x"], s["codes"], s["scale"], bias=True)
        rows = torch.arange(300, device="cuda") != 20
        assert torch.equal(dx[rows], want[0][rows]) and not dx[20].isfinite().any()
        k, n = torch.arange(256, device="cuda") != 9, torch.arange(144, device="cuda") != 30
        assert not dw[9].isfinite().any() and not dw[:, 30].isfinite().any() and not db[30].isfinite()
        assert torch.equal(dw[k][:, n], want[1][k][:, n]) and torch.equal(db[n], want[2][n])


def test_more_tiles_of_rows_than_a_grid_has_in_its_second_dimension():
    """65537 tiles of 128 rows through a narrow weight, offsets past 2^31; all gradients."""
    tokens, rows, cols = 65536 * 128 + 77, 272, 16
    s = make(1, rows, cols, False, 5)
    g = M.gen(6)
    x = torch.randn((tokens, rows), generator=g, device="cuda", dtype=BF16)
    dy = torch.randn((tokens, cols), generator=g, device="cuda", dtype=BF16)
    y = ops.linear(x, s["codes"], s["scale"])
    dx, dw, db = ops.linear_grad(dy, x, s["codes"], s["scale"], bias=True)
    edges = [0, 65535 * 128, 2**31 // 384, 2**31 // rows, tokens - 300]
    want_w, want_b = torch.zeros((rows, cols), dtype=torch.float64, device="cuda"), 0.0
    for i in range(0, tokens, 1 << 19):
        d = dy[i:i + (1 << 19)].double()
        want_w += x[i:i + (1 << 19)].double().T @ d
        want_b = want_b + d.sum(0)
    for i in edges:
        at = slice(max(i - 200, 0), i + 300)
        v, d = x[at].double(), dy[at].double()
        check(y[at], v @ s["w"], v.abs() @ s["w"].abs(), BF16)
        check(dx[at], d @ s["w"].T, d.abs() @ s["w"].T.abs(), BF16)
    # 32769 additions of 256 rows' sums round by 2^-24 of the sum so far, of either sign: 181 * 2^-24 = 1.1e-5 of the norm
    assert rel(dw, want_w) <= 2e-5 and rel(db, want_b) <= 2e-5


@pytest.mark.parametrize("transposed", [False, True])
def test_no_tokens(transposed):
    s = make(0, 64, 32, transposed, 1)
    y, pre = ops.linear(s["x"], s["codes"], s["scale"], transposed=transposed, activation="silu", save=True)
    assert y.shape == (0, 64 if transposed else 32)
    dx, dw, db = ops.linear_grad(s["dy"], s["x"], s["codes"], s["scale"], transposed=transposed, activation="silu", pre=pre, bias=True)
    assert dx.shape == s["x"].shape and not dw.any() and not db.any()
