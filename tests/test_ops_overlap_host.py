"""Results over what a call still reads are refused: no GPU.

Device pointers are stand-ins (host memory): a call that the library refuses touches none of them."""
import ctypes as C

import numpy as np
import pytest

from blockwise_fp8_zero_fold_gb300 import build as fp8build
from blockwise_fp8_zero_fold_gb300 import fp8z1 as F


@pytest.fixture(scope="module", autouse=True)
def built():
    fp8build.build()
    return F.lib()


_MEM = np.zeros(1 << 22, np.uint8)
P = (_MEM.ctypes.data + 255) & ~255  # 256-byte aligned
AT = [P + (i << 18) for i in range(15)]  # 256 KB apart: buffers that share nothing

# 40 rows through a weight of 64 x 64
DIMS = dict(tokens=40, rows=64, cols=64, transposed=0, activation=F.ACT_NONE, x_type=F.BF16, y_type=F.BF16)
X, XS, CODES, SCALES, BIAS, RES, Y, PRE, WS, DY, DX, DW, DB = AT[:13]
LINEAR = dict(x=X, ld_x=64, xs=XS, codes=CODES, scales=SCALES, bias=BIAS, r=RES, ld_r=64, y=Y, ld_y=64, pre=PRE, ws=WS, stream=None)
FP8, F32, SILU = dict(x_type=F.E4M3), dict(y_type=F.F32), dict(activation=F.ACT_SILU)


@pytest.mark.parametrize("dims,change", [
    ({}, dict(pre=Y)), ({}, dict(pre=Y + 40 * 64 * 2 - 4)), ({}, dict(pre=RES)), ({}, dict(y=RES + 128)), ({}, dict(y=RES - 128)),
    ({}, dict(y=RES, ld_y=72)), ({}, dict(y=RES + 64, ld_y=128, ld_r=128)), (F32, dict(y=RES)), (F32, dict(y=RES + 64)),
    ({}, dict(y=CODES)), ({}, dict(y=CODES - 64)), ({}, dict(y=SCALES)), ({}, dict(y=BIAS + 64)), ({}, dict(pre=CODES)),
    ({}, dict(pre=BIAS)), (FP8, dict(y=X)), (FP8, dict(y=X + 1024)), (FP8, dict(y=XS)), (FP8, dict(pre=XS))])
def test_product(dims, change):
    d = F.fp8z1_linear_dims(*{**DIMS, **dims}.values())
    assert F.lib().fp8z1_linear(C.byref(d), *{**LINEAR, **change}.values()) == F.EINVAL


LGRAD = dict(dy=DY, ld_dy=64, x=X, ld_x=64, codes=CODES, scales=SCALES, pre=PRE, dx=DX, ld_dx=64, dw=DW, db=DB, ws=WS, stream=None)


@pytest.mark.parametrize("dims,change", [
    ({}, dict(dx=X)), ({}, dict(dx=X + 128)), ({}, dict(dx=DY)), ({}, dict(dx=DY - 2)), (SILU, dict(dx=X)), (F32, dict(dx=X)),
    ({}, dict(dw=DX)), ({}, dict(dx=DW + 64 * 64 * 4 - 2)), ({}, dict(db=DW + 64)), ({}, dict(db=DX)), ({}, dict(dw=X)),
    ({}, dict(dw=DY)), ({}, dict(dx=CODES)), ({}, dict(dx=SCALES)), ({}, dict(dx=CODES, dw=None))])
def test_products_gradients(dims, change):
    d = F.fp8z1_linear_dims(*{**DIMS, **dims}.values())
    assert F.lib().fp8z1_linear_grad(C.byref(d), *{**LGRAD, **change}.values()) == F.EINVAL


NORM = dict(rows=40, dim=64, x=X, type=F.BF16, ld_x=64, r=RES, ld_r=64, w=BIAS, eps=1e-6, total=DX, ld_t=64, y=Y, ld_y=64, codes=CODES,
            scales=SCALES, stream=None)


@pytest.mark.parametrize("change", [
    dict(total=Y), dict(total=Y + 128), dict(total=X + 128), dict(y=X + 128), dict(y=X - 2), dict(total=RES + 2),
    dict(y=RES - 64 * 2 * 39), dict(y=X, ld_y=72), dict(total=RES, ld_r=72), dict(y=X + 64, ld_x=128, ld_y=128), dict(codes=X),
    dict(codes=RES + 64), dict(codes=Y), dict(codes=DX), dict(scales=X), dict(scales=CODES + 64), dict(scales=Y), dict(y=BIAS),
    dict(total=BIAS), dict(codes=BIAS), dict(scales=BIAS + 32)])
def test_norm(change):
    assert F.lib().fp8z1_rms_norm(*{**NORM, **change}.values()) == F.EINVAL


GRAD = dict(rows=40, dim=64, dy=DY, type=F.BF16, ld_dy=64, s=X, ld_s=64, w=BIAS, eps=1e-6, dt=RES, ld_dt=64, dx=DX, ld_dx=64, dw=DB, ws=WS,
            stream=None)


@pytest.mark.parametrize("change", [
    dict(dx=DY + 128), dict(dx=DY, ld_dx=72), dict(dx=X - 128), dict(dx=X, ld_s=80), dict(dx=RES + 2), dict(dx=RES, ld_dt=128),
    dict(dx=BIAS), dict(dx=DB - 64)])
def test_norms_gradient(change):
    assert F.lib().fp8z1_rms_norm_grad(*{**GRAD, **change}.values()) == F.EINVAL


ROUTE = dict(ids=X, id_bytes=4, tokens=40, top=2, experts=8, offsets=SCALES, place=Y, stream=None)


@pytest.mark.parametrize("change", [
    dict(place=X), dict(place=X + 316), dict(id_bytes=8, place=X + 320), dict(offsets=X + 64), dict(offsets=Y + 16), dict(place=SCALES + 32),
    dict(place=SCALES - 316)])
def test_route(change):
    assert F.lib().fp8z1_route(*{**ROUTE, **change}.values()) == F.EINVAL


DISPATCH = dict(tokens=40, top=2, experts=8, dim=64, x=X, type=F.BF16, ld_x=64, offsets=SCALES, place=BIAS, rows=Y, ld_rows=64, stream=None)


@pytest.mark.parametrize("change", [
    dict(rows=X), dict(rows=X + 128 * 39), dict(rows=X - 128 * 79), dict(rows=X + 128, ld_x=96, ld_rows=96), dict(rows=SCALES),
    dict(rows=BIAS + 64)])
def test_dispatch(change):
    assert F.lib().fp8z1_dispatch(*{**DISPATCH, **change}.values()) == F.EINVAL


COMBINE = dict(tokens=40, top=2, dim=64, rows=X, type=F.BF16, ld_rows=64, place=BIAS, w=DW, r=RES, ld_r=64, y=Y, ld_y=64, stream=None)


@pytest.mark.parametrize("change", [
    dict(y=X), dict(y=X + 40 * 128), dict(y=X + 79 * 128), dict(y=X - 39 * 128), dict(y=RES + 128), dict(y=RES, ld_r=72), dict(y=BIAS),
    dict(y=DW + 64)])
def test_combine(change):
    assert F.lib().fp8z1_combine(*{**COMBINE, **change}.values()) == F.EINVAL


CGRAD = dict(tokens=40, top=2, experts=8, dim=64, dy=DY, type=F.BF16, ld_dy=64, rows=X, ld_rows=64, offsets=SCALES, place=BIAS, w=DW, d=DX,
             ld_d=64, dw=DB, stream=None)


@pytest.mark.parametrize("change", [
    dict(d=DY), dict(d=DY + 39 * 128), dict(d=DY - 79 * 128), dict(d=X + 128), dict(d=X, ld_rows=72), dict(d=BIAS), dict(d=DW), dict(d=DB),
    dict(d=SCALES), dict(dw=DY), dict(dw=X + 64), dict(dw=BIAS), dict(dw=SCALES), dict(dw=DW + 4)])
def test_combines_gradient(change):
    assert F.lib().fp8z1_combine_grad(*{**CGRAD, **change}.values()) == F.EINVAL
