"""Root-mean-square norm, its 8-bit form and its gradient, against their definition in 64 bits."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6

# FP32 arithmetic beside the one rounding: a sum of squares of up to 2^14 terms in threads and a tree (32 + 11 additions
# in a row: 43 half steps of 2^-24, half of them through the square root), and a handful of products: 2^-24 * 32 = 2^-19.
SUMS = 2.0**-19


def check(got, want, dtype, mag=None):
    """One rounding to the type, and FP32 sums relative to the terms."""
    err = (got.double() - want).abs()
    tol = M.half_step(dtype) * want.abs() * 1.01 + SUMS * (want.abs() if mag is None else mag + want.abs()) + 1e-37
    assert (err <= tol).all(), float((err / tol).max())


def make(rows, dim, dtype, seed, by=1.0):
    g = M.gen(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return ((r(rows, dim) * by).to(dtype), (r(rows, dim) * 3 * by).to(dtype), r(dim) * 0.3 + 1.0, r(rows, dim).to(dtype),
            r(rows, dim).to(dtype))


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 64), (2, 127), (2, 128), (2, 129), (9, 255), (8, 256), (17, 257), (64, 1000), (33, 1024),
          (2, 1025), (7, 2048), (700, 520), (1, 7168), (2500, 304), (5, 4097), (3, 8192), (2, 8200), (2, 16384), (2, 16383),
          (400, 7168), (5000, 72), (1300, 2049), (1900, 1032), (650, 8200), (620, 16383), (1500, 7168), (3000, 1100)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_norm(rows, dim, dtype):
    x, r, w, dy, dt = make(rows, dim, dtype, rows * 7 + dim)
    y = ops.rms_norm(x, w, eps=EPS)
    check(y, M.norm(x, w, EPS)["y"], dtype)
    y, total = ops.rms_norm(x, w, residual=r, eps=EPS)
    want = M.norm(x, w, EPS, r)
    assert torch.equal(total, (x.float() + r.float()).to(dtype))
    check(y, M.norm(total, w, EPS)["y"], dtype)
    assert torch.equal(total.double(), want["total"].double()) or dtype == BF16


def values(codes, scale, dim):
    return codes.to(torch.float64) * scale.double().repeat_interleave(128, 1)[:, :dim]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_norm_in_8_bits(rows, dim, dtype):
    x, r, w, _, _ = make(rows, dim, dtype, rows * 7 + dim + 1)
    codes, scale, total = ops.rms_norm_fp8(x, w, residual=r, eps=EPS)
    y = M.norm(total, w, EPS)["y"]
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == x.shape and scale.shape == (rows, -(-dim // 128))
    for b in range(scale.shape[1]):
        some = slice(b * 128, min(dim, b * 128 + 128))
        top = y[:, some].abs().amax(1)
        # the scale: FP32 arithmetic of the largest, one division
        assert ((scale[:, b].double() - top / 448).abs() <= 2 * SUMS * top / 448 + 1e-44).all()
        s = scale[:, b].double()[:, None]
        # a code is off by half a step of its binade (2^-4 of the value), at least of the smallest step 2^-9
        err = (codes[:, some].double() * s - y[:, some]).abs()
        assert (err <= (2.0**-4 * y[:, some].abs()).clamp(min=2.0**-10 * s) * (1 + 2.0**-10) + SUMS * y[:, some].abs()).all()
        # the largest of each 128 is at the top of the range
        assert (codes[:, some].double().abs().amax(1) == 448).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_gradient(rows, dim, dtype):
    x, r, w, dy, dt = make(rows, dim, dtype, rows * 7 + dim + 2)
    for d_total in (None, dt):
        dx, dw = ops.rms_norm_grad(dy, x, w, eps=EPS, d_total=d_total)
        want = M.norm(x, w, EPS, None, dy, d_total)
        check(dx, want["dx"], dtype, want["dx_mag"])
        # sums of up to 5000 rows in 300 CTAs: 17 + 10 + 5 additions in a row, rstd beside them
        assert ((dw.double() - want["d_weight"]).abs() <= 2.0**-18 * want["d_weight_mag"] + 1e-37).all()
        again = ops.rms_norm_grad(dy, x, w, eps=EPS, d_total=d_total)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim", [(1000, 3840), (1000, 3841), (901, 4096), (1201, 4097), (700, 4863), (700, 4864), (700, 4865),
                                      (640, 7169), (900, 7680), (610, 7681)])
def test_gradient_of_widths_that_take_other_threads(rows, dim, dtype):
    """One row of a CTA under way or two, and widths on both sides."""
    test_gradient(rows, dim, dtype)


def test_gradient_against_differences():
    x, _, w, dy, _ = make(3, 200, F32, 5)
    dx, dw = ops.rms_norm_grad(dy, x, w, eps=EPS)
    f = lambda x, w: float((dy.double() * M.norm(x, w, EPS)["y"]).sum())  # noqa: E731
    for i, j in ((0, 0), (1, 77), (2, 199)):
        h = torch.zeros_like(x, dtype=torch.float64)
        h[i, j] = 1e-5
        d = (f(x.double() + h, w) - f(x.double() - h, w)) / 2e-5
        assert abs(float(dx[i, j]) - d) <= 1e-4 * max(1.0, abs(d))
    for j in (0, 128, 199):
        h = torch.zeros_like(w, dtype=torch.float64)
        h[j] = 1e-5
        d = (f(x, w.double() + h) - f(x, w.double() - h)) / 2e-5
        assert abs(float(dw[j]) - d) <= 1e-4 * max(1.0, abs(d))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,at", [(8, 0), (3, 0), (1, 1), (0, 1), (16, 8)])
@pytest.mark.parametrize("dim", [96, 264, 2056])
def test_strides_and_offsets(dim, pad, at, dtype):
    x, r, w, dy, dt = make(6, dim, dtype, dim + pad)
    xs, rs, dys, dts = (M.strided(t, pad, at) for t in (x, r, dy, dt))
    outs = [M.strided(torch.zeros_like(x), pad, at) for _ in range(3)]
    y, total = ops.rms_norm(xs, w, residual=rs, eps=EPS, out=outs[0], total=outs[1])
    assert y is outs[0] and total is outs[1]
    check(y, M.norm(total, w, EPS)["y"], dtype)
    assert torch.equal(total, (x.float() + r.float()).to(dtype))
    dx, dw = ops.rms_norm_grad(dys, total, w, eps=EPS, d_total=dts, dx=outs[2])
    want = M.norm(total, w, EPS, None, dy, dt)
    check(dx, want["dx"], dtype, want["dx_mag"])
    if pad:  # between the rows nothing is written
        for o in outs:
            gaps = o.as_strided((5, pad), (dim + pad, 1), o.storage_offset() + dim)
            assert gaps.isnan().all()


def test_weight_of_another_alignment():
    x, _, w, dy, _ = make(4, 512, BF16, 3)
    odd = torch.cat([w[:1], w])[1:]
    assert odd.data_ptr() % 16
    check(ops.rms_norm(x, odd, eps=EPS), M.norm(x, w, EPS)["y"], BF16)
    dx, _ = ops.rms_norm_grad(dy, x, odd, eps=EPS)
    want = M.norm(x, w, EPS, None, dy)
    check(dx, want["dx"], BF16, want["dx_mag"])


@pytest.mark.parametrize("dim", [40, 1536, 2001])
def test_in_place(dim):
    x, r, w, dy, dt = make(50, dim, BF16, dim)
    y, total = ops.rms_norm(x, w, residual=r, eps=EPS)
    a, b = x.clone(), r.clone()
    y2, t2 = ops.rms_norm(a, w, residual=b, eps=EPS, out=a, total=b)
    assert y2 is a and t2 is b and torch.equal(a, y) and torch.equal(b, total)
    dx, dw = ops.rms_norm_grad(dy, total, w, eps=EPS, d_total=dt)
    for k in range(2):
        d, t = dy.clone(), dt.clone()
        got = ops.rms_norm_grad(d, total, w, eps=EPS, d_total=t, dx=(d, t)[k])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("dim", [24, 1200, 2050])
def test_ends_of_the_range(dim):
    """Squares beyond FP32, rows of zeros, one infinity, one NaN: no row touches another."""
    x, _, w, dy, _ = make(6, dim, F32, dim)
    x[1] *= 1e30
    x[2] = 0
    x[3, dim // 2] = float("inf")
    x[4, dim // 2] = float("nan")
    x[5] *= 1e-30
    y = ops.rms_norm(x, w, eps=EPS)
    dx, dw = ops.rms_norm_grad(dy, x, w, eps=EPS)
    want = M.norm(x, w, EPS, None, dy)
    for k in (0, 1, 2, 5):
        check(y[k], want["y"][k], F32)
        check(dx[k], want["dx"][k], F32, want["dx_mag"][k])
    assert y[3, dim // 2].isnan() and not y[3, : dim // 2].any() and y[4].isnan().all()
    some = [0, 1, 2, 5]
    _, dw = ops.rms_norm_grad(dy[some], x[some], w, eps=EPS)
    assert ((dw.double() - M.norm(x[some], w, EPS, None, dy[some])["d_weight"]).abs() <= 1e-4).all()
    codes, scale = ops.rms_norm_fp8(x, w, eps=EPS)
    assert (scale[2] == 1).all() and not codes[2].float().any()
    assert codes[4].float().isnan().all() and codes[:3].float().isfinite().all() and codes[5].float().isfinite().all()


def test_tiny_results_in_8_bits():
    """128 numbers below 2^-117 are 0, with a scale of 1; from there on they are held."""
    x = torch.ones(2, 384, device="cuda")
    w = torch.ones(384, device="cuda")
    for tiny in (1e-44, 1e-38, 2.0**-117.1):
        w[:128], w[256:] = tiny, 2.0**-116.9
        codes, scale = ops.rms_norm_fp8(x, w)
        assert (scale[:, 0] == 1).all() and not codes[:, :128].float().any() and (codes[:, 128:].float() == 448).all()
        y = M.norm(x, w, EPS)["y"][:, 256:]
        assert ((scale[:, 2:].double() * 448 - y).abs() <= 2.0**-21 * y).all()


@pytest.mark.parametrize("shape", [(0, 64), (2, 0, 64), (2, 3, 64), (64,)])
def test_shapes(shape):
    g = M.gen(1)
    x, w = torch.randn(shape, generator=g, device="cuda"), torch.ones(64, device="cuda")
    y, total = ops.rms_norm(x, w, residual=x)
    assert y.shape == total.shape == x.shape
    codes, scale = ops.rms_norm_fp8(x, w)
    assert codes.shape == x.shape and scale.shape == x.shape[:-1] + (1,)
    dx, dw = ops.rms_norm_grad(x, x, w)
    assert dx.shape == x.shape and dw.shape == (64,)
    if x.numel() == 0:
        assert not dw.any()
    else:
        check(y, M.norm(2 * x, w, EPS)["y"], F32)


def test_many_rows():
    """More than 2^31 elements: offsets pass 32 bits."""
    n, dim = 300_000, 7176
    x = torch.zeros(n, dim, dtype=BF16, device="cuda")
    x[-3:] = torch.randn(3, dim, generator=M.gen(2), device="cuda").to(BF16)
    w = torch.ones(dim, device="cuda")
    y = ops.rms_norm(x, w, eps=EPS)
    check(y[-3:], M.norm(x[-3:], w, EPS)["y"], BF16)
    assert not y[:10].any()
    dx, dw = ops.rms_norm_grad(x, x, w, eps=EPS)
    want = M.norm(x[-3:], w, EPS, None, x[-3:])
    check(dx[-3:], want["dx"], BF16, want["dx_mag"])
    assert ((dw.double() - want["d_weight"]).abs() <= 2.0**-18 * want["d_weight_mag"]).all()
