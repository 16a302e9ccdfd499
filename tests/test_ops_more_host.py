"""What the norm, the routing and the matrix product refuse, and the host side of their sizes: no GPU.

Device pointers are stand-ins (host memory): a call that the library refuses touches none of them."""
import ctypes as C

import numpy as np
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import build as fp8build
from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops
from tests.test_ops_streams_host import Stream, world  # noqa: F401


@pytest.fixture(scope="module", autouse=True)
def built():
    fp8build.build()
    return F.lib()


_MEM = np.zeros(4096, np.uint8)
P = (_MEM.ctypes.data + 255) & ~255  # 256-byte aligned
NAN, INF = float("nan"), float("inf")


def status(name, args):
    return getattr(F.lib(), name)(*args.values())


NORM = dict(rows=2, dim=64, x=P, type=F.BF16, ld_x=64, r=P, ld_r=64, w=P, eps=1e-6, total=P, ld_t=64, y=P + 1024, ld_y=64, codes=P,
            scales=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), F.EINVAL), (dict(rows=(1 << 30) + 1), F.EINVAL), (dict(dim=0), F.EINVAL), (dict(dim=16385), F.EINVAL),
    (dict(type=2), F.EINVAL), (dict(type=-1), F.EINVAL), (dict(x=None), F.EINVAL), (dict(w=None), F.EINVAL),
    (dict(ld_x=63), F.EINVAL), (dict(ld_r=8), F.EINVAL), (dict(ld_t=63), F.EINVAL), (dict(ld_y=0), F.EINVAL),
    (dict(total=None), F.EINVAL), (dict(r=None), F.EINVAL), (dict(codes=None), F.EINVAL), (dict(scales=None), F.EINVAL),
    (dict(y=None, codes=None, scales=None), F.EINVAL), (dict(eps=0.0), F.EINVAL), (dict(eps=-1.0), F.EINVAL),
    (dict(eps=NAN), F.EINVAL), (dict(eps=INF), F.EINVAL), (dict(eps=1e-30), F.EINVAL), (dict(x=P + 1), F.EALIGN),
    (dict(r=P + 1), F.EALIGN), (dict(total=P + 1), F.EALIGN), (dict(y=P + 1), F.EALIGN), (dict(w=P + 2), F.EALIGN),
    (dict(scales=P + 2), F.EALIGN), (dict(type=F.F32, x=P + 2), F.EALIGN), (dict(y=P), F.EINVAL),  # y over the sum
    (dict(rows=0, x=None, w=None, r=None, total=None, y=None, codes=None, scales=None), F.OK)])
def test_norm_refusals(change, want):
    assert status("fp8z1_rms_norm", {**NORM, **change}) == want


GRAD = dict(rows=2, dim=64, dy=P, type=F.BF16, ld_dy=64, s=P, ld_s=64, w=P, eps=1e-6, dt=P, ld_dt=64, dx=P, ld_dx=64, dw=P, ws=P,
            stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), F.EINVAL), (dict(dim=16385), F.EINVAL), (dict(type=3), F.EINVAL), (dict(dy=None), F.EINVAL),
    (dict(s=None), F.EINVAL), (dict(w=None), F.EINVAL), (dict(dx=None), F.EINVAL), (dict(dw=None), F.EINVAL),
    (dict(ws=None), F.EINVAL), (dict(ld_dy=1), F.EINVAL), (dict(ld_s=63), F.EINVAL), (dict(ld_dt=63), F.EINVAL),
    (dict(ld_dx=63), F.EINVAL), (dict(eps=0.0), F.EINVAL), (dict(dy=P + 1), F.EALIGN), (dict(s=P + 1), F.EALIGN),
    (dict(dt=P + 1), F.EALIGN), (dict(dx=P + 1), F.EALIGN), (dict(dw=P + 2), F.EALIGN), (dict(w=P + 1), F.EALIGN),
    (dict(ws=P + 16), F.EALIGN), (dict(rows=0, dw=None), F.EINVAL)])
def test_norm_grad_refusals(change, want):
    assert status("fp8z1_rms_norm_grad", {**GRAD, **change}) == want


ROUTE = dict(ids=P, id_bytes=4, tokens=4, top=2, experts=8, offsets=P, place=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(ids=None), F.EINVAL), (dict(id_bytes=2), F.EINVAL), (dict(tokens=-1), F.EINVAL), (dict(top=0), F.EINVAL),
    (dict(top=65), F.EINVAL), (dict(experts=0), F.EINVAL), (dict(experts=1025), F.EINVAL), (dict(offsets=None), F.EINVAL),
    (dict(place=None), F.EINVAL), (dict(tokens=1 << 30, top=2), F.EINVAL), (dict(ids=P + 4, id_bytes=8), F.EALIGN),
    (dict(offsets=P + 2), F.EALIGN), (dict(place=P + 1), F.EALIGN)])
def test_route_refusals(change, want):
    assert status("fp8z1_route", {**ROUTE, **change}) == want


DISPATCH = dict(tokens=4, top=2, experts=8, dim=64, x=P, type=F.BF16, ld_x=64, offsets=P, place=P, rows=P, ld_rows=64, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(tokens=-1), F.EINVAL), (dict(top=0), F.EINVAL), (dict(experts=0), F.EINVAL), (dict(dim=0), F.EINVAL),
    (dict(dim=(1 << 23) + 1, ld_x=1 << 24, ld_rows=1 << 24), F.EINVAL), (dict(type=2), F.EINVAL), (dict(x=None), F.EINVAL),
    (dict(offsets=None), F.EINVAL), (dict(place=None), F.EINVAL), (dict(rows=None), F.EINVAL), (dict(ld_x=63), F.EINVAL),
    (dict(ld_rows=63), F.EINVAL), (dict(x=P + 1), F.EALIGN), (dict(rows=P + 1), F.EALIGN), (dict(offsets=P + 1), F.EALIGN),
    (dict(place=P + 2), F.EALIGN), (dict(type=F.F32, x=P + 2), F.EALIGN),
    (dict(tokens=0, x=None, offsets=None, place=None, rows=None), F.OK)])
def test_dispatch_refusals(change, want):
    assert status("fp8z1_dispatch", {**DISPATCH, **change}) == want


COMBINE = dict(tokens=4, top=2, dim=64, rows=P, type=F.BF16, ld_rows=64, place=P, w=P, r=P, ld_r=64, y=P, ld_y=64, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(tokens=-1), F.EINVAL), (dict(top=65), F.EINVAL), (dict(dim=0), F.EINVAL), (dict(type=2), F.EINVAL),
    (dict(rows=None), F.EINVAL), (dict(place=None), F.EINVAL), (dict(y=None), F.EINVAL), (dict(ld_rows=63), F.EINVAL),
    (dict(ld_r=63), F.EINVAL), (dict(ld_y=63), F.EINVAL), (dict(rows=P + 1), F.EALIGN), (dict(r=P + 1), F.EALIGN),
    (dict(y=P + 1), F.EALIGN), (dict(place=P + 1), F.EALIGN), (dict(w=P + 2), F.EALIGN), (dict(tokens=0, rows=None, y=None), F.OK)])
def test_combine_refusals(change, want):
    assert status("fp8z1_combine", {**COMBINE, **change}) == want


CGRAD = dict(tokens=4, top=2, experts=8, dim=64, dy=P, type=F.BF16, ld_dy=64, rows=P, ld_rows=64, offsets=P, place=P, w=P, d=P,
             ld_d=64, dw=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(tokens=-1), F.EINVAL), (dict(experts=1025), F.EINVAL), (dict(dim=0), F.EINVAL), (dict(type=2), F.EINVAL),
    (dict(dy=None), F.EINVAL), (dict(rows=None), F.EINVAL), (dict(offsets=None), F.EINVAL), (dict(place=None), F.EINVAL),
    (dict(w=None), F.EINVAL), (dict(d=None), F.EINVAL), (dict(dw=None), F.EINVAL), (dict(ld_dy=63), F.EINVAL),
    (dict(ld_rows=63), F.EINVAL), (dict(ld_d=63), F.EINVAL), (dict(dy=P + 1), F.EALIGN), (dict(rows=P + 1), F.EALIGN),
    (dict(d=P + 1), F.EALIGN), (dict(dw=P + 2), F.EALIGN), (dict(w=P + 1), F.EALIGN), (dict(offsets=P + 2), F.EALIGN),
    (dict(place=P + 2), F.EALIGN)])
def test_combine_grad_refusals(change, want):
    assert status("fp8z1_combine_grad", {**CGRAD, **change}) == want


@pytest.mark.parametrize("name,args,out,given", [("fp8z1_dispatch", DISPATCH, "rows", "x"), ("fp8z1_combine", COMBINE, "y", "rows"),
                                                 ("fp8z1_combine_grad", CGRAD, "d", "dy")])
def test_rows_go_to_rows_of_their_own(name, args, out, given):
    """Tokens would read what others have written, were the result its own input."""
    assert args[out] == args[given] and status(name, args) == F.EINVAL


DIMS = dict(tokens=4, rows=64, cols=32, transposed=0, activation=F.ACT_NONE, x_type=F.BF16, y_type=F.BF16)


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(rows=0), dict(rows=(1 << 22) + 1), dict(cols=0), dict(cols=8), dict(cols=24),
    dict(cols=(1 << 22) + 16), dict(transposed=2), dict(transposed=-1), dict(activation=3), dict(activation=-1), dict(x_type=F.F32),
    dict(x_type=3), dict(y_type=F.E4M3), dict(y_type=-1)])
def test_linear_dims_refused(change):
    with pytest.raises(F.Fp8z1Error) as e:
        F.fp8z1_linear_sizes(F.fp8z1_linear_dims(*{**DIMS, **change}.values()))
    assert e.value.status == F.EINVAL


def test_sizes():
    n = C.c_int64(-7)
    assert F.lib().fp8z1_linear_sizes(None, C.byref(n), C.byref(n)) == F.EINVAL and n.value == -7
    d = F.fp8z1_linear_dims(*DIMS.values())
    assert F.lib().fp8z1_linear_sizes(C.byref(d), None, C.byref(n)) == F.EINVAL
    small = F.fp8z1_linear_sizes(d)
    large = F.fp8z1_linear_sizes(F.fp8z1_linear_dims(*{**DIMS, "tokens": 400}.values()))
    assert all(0 < a <= b for a, b in zip(small, large))
    assert F.fp8z1_linear_sizes(F.fp8z1_linear_dims(*{**DIMS, "x_type": F.E4M3}.values()))[0] == 0
    # the largest sizes do not wrap
    assert all(v > 0 for v in F.fp8z1_linear_sizes(F.fp8z1_linear_dims(1 << 30, 1 << 22, 1 << 22, 0, 1, F.BF16, F.F32)))
    assert F.lib().fp8z1_rms_norm_grad_workspace(2, 0, C.byref(n)) == F.EINVAL
    assert F.lib().fp8z1_rms_norm_grad_workspace(2, 8, None) == F.EINVAL
    assert 0 < F.fp8z1_rms_norm_grad_workspace(1, 64) <= F.fp8z1_rms_norm_grad_workspace(1000, 64)
    assert F.fp8z1_rms_norm_grad_workspace(1 << 30, 16384) > 0


LINEAR = dict(x=P, ld_x=64, xs=P, codes=P, scales=P, bias=P, r=P, ld_r=32, y=P, ld_y=32, pre=P, ws=P, stream=None)
FP8 = dict(x_type=F.E4M3)


@pytest.mark.parametrize("dims,change,want", [
    ({}, dict(x=None), F.EINVAL), ({}, dict(codes=None), F.EINVAL), ({}, dict(scales=None), F.EINVAL), ({}, dict(y=None), F.EINVAL),
    ({}, dict(ws=None), F.EINVAL), (FP8, dict(xs=None), F.EINVAL), ({}, dict(ld_x=63), F.EINVAL), ({}, dict(ld_y=31), F.EINVAL),
    ({}, dict(ld_r=31), F.EINVAL), (dict(transposed=1), dict(ld_y=63), F.EINVAL), (dict(cols=20), {}, F.EINVAL),
    ({}, dict(x=P + 1), F.EALIGN), (FP8, dict(x=P + 8), F.EALIGN), (FP8, dict(ld_x=72), F.EALIGN), ({}, dict(codes=P + 8), F.EALIGN),
    ({}, dict(scales=P + 2), F.EALIGN), ({}, dict(bias=P + 2), F.EALIGN), ({}, dict(r=P + 1), F.EALIGN), ({}, dict(y=P + 1), F.EALIGN),
    (dict(y_type=F.F32), dict(y=P + 2), F.EALIGN), ({}, dict(pre=P + 2), F.EALIGN), ({}, dict(ws=P + 16), F.EALIGN),
    (FP8, dict(xs=P + 2), F.EALIGN), (dict(tokens=0), dict(x=None, y=None, ws=None), F.OK)])
def test_linear_refusals(dims, change, want):
    d = F.fp8z1_linear_dims(*{**DIMS, **dims}.values())
    assert F.lib().fp8z1_linear(C.byref(d), *{**LINEAR, **change}.values()) == want


def test_linear_null_dims():
    assert F.lib().fp8z1_linear(None, *LINEAR.values()) == F.EINVAL
    assert F.lib().fp8z1_linear_grad(None, *LGRAD.values()) == F.EINVAL
    assert F.lib().fp8z1_linear_timeouts(None) == F.EINVAL
    assert F.lib().fp8z1_checked_linear_stall(1) == F.EINVAL  # a release build


LGRAD = dict(dy=P, ld_dy=32, x=P, ld_x=64, codes=P, scales=P, pre=P, dx=P, ld_dx=64, dw=P, db=P, ws=P, stream=None)
SILU = dict(activation=F.ACT_SILU)


@pytest.mark.parametrize("dims,change,want", [
    (FP8, {}, F.EINVAL), ({}, dict(dx=None, dw=None, db=None), F.EINVAL), ({}, dict(dy=None), F.EINVAL), ({}, dict(x=None), F.EINVAL),
    ({}, dict(codes=None), F.EINVAL), ({}, dict(scales=None), F.EINVAL), ({}, dict(ws=None), F.EINVAL), (SILU, dict(pre=None), F.EINVAL),
    ({}, dict(ld_dy=31), F.EINVAL), ({}, dict(ld_x=63), F.EINVAL), ({}, dict(ld_dx=63), F.EINVAL), ({}, dict(dy=P + 1), F.EALIGN),
    (dict(y_type=F.F32), dict(dy=P + 2), F.EALIGN), ({}, dict(x=P + 1), F.EALIGN), ({}, dict(dx=P + 1), F.EALIGN),
    ({}, dict(dw=P + 8), F.EALIGN), ({}, dict(db=P + 2), F.EALIGN), ({}, dict(codes=P + 4), F.EALIGN), ({}, dict(ws=P + 128), F.EALIGN),
    (SILU, dict(pre=P + 2), F.EALIGN)])
def test_linear_grad_refusals(dims, change, want):
    d = F.fp8z1_linear_dims(*{**DIMS, **dims}.values())
    assert F.lib().fp8z1_linear_grad(C.byref(d), *{**LGRAD, **change}.values()) == want


def tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    codes, scale = torch.zeros(64, 32, dtype=torch.uint8), torch.ones(1, 1)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    r = ops.Route(torch.zeros(9, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32))
    return x, w, codes, scale, ids, r, torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(4, 2)


@pytest.mark.parametrize("call", [
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x, w),                                   # not on a GPU
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x.half(), w),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x, w.bfloat16()),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x, w[:32]),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x.t(), torch.ones(4)),                   # columns, not rows
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x.reshape(2, 2, 64).transpose(0, 1), w),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x[:1].expand(4, 64), w),                 # rows on top of each other
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm_fp8(x.float().half(), w),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm_grad(x, x, w[:3]),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm_grad(x, x.half(), w),
    lambda x, w, c, s, i, r, rows, cw: ops.route(i, 8),
    lambda x, w, c, s, i, r, rows, cw: ops.route(i.float(), 8),
    lambda x, w, c, s, i, r, rows, cw: ops.route(i.t(), 8),
    lambda x, w, c, s, i, r, rows, cw: ops.route(i[None], 8),
    lambda x, w, c, s, i, r, rows, cw: ops.dispatch(x[:3], r),
    lambda x, w, c, s, i, r, rows, cw: ops.dispatch(x.half(), r),
    lambda x, w, c, s, i, r, rows, cw: ops.dispatch(x, ops.Route(r.offsets.long(), r.place)),
    lambda x, w, c, s, i, r, rows, cw: ops.dispatch(x, ops.Route(r.offsets, r.place.t())),
    lambda x, w, c, s, i, r, rows, cw: ops.combine(rows[:7], r),
    lambda x, w, c, s, i, r, rows, cw: ops.combine(rows, r, cw.double()),
    lambda x, w, c, s, i, r, rows, cw: ops.combine(rows, r, cw[:3]),
    lambda x, w, c, s, i, r, rows, cw: ops.combine_grad(x, rows[:5], r, cw),
    lambda x, w, c, s, i, r, rows, cw: ops.combine_grad(x, rows, r, cw.t()),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s),                                  # not on a GPU
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x[:, :32], c, s),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x.float(), c, s),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s, activation="relu"),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s, dtype=torch.float16),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c[None].repeat(2, 1, 1), s[None].repeat(2, 1, 1)),  # several experts
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s.repeat(2, 1)),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s, transposed=True),
    lambda x, w, c, s, i, r, rows, cw: ops.linear_grad(x, x, c, s),
    lambda x, w, c, s, i, r, rows, cw: ops.linear_grad(x[:, :32], x, c, s, activation="silu"),
    lambda x, w, c, s, i, r, rows, cw: ops.linear_grad(x[:, :32], x.view(torch.uint8)[:, :64], c, s),
])
def test_tensors_that_do_not_fit(call):
    """ops.py's own checks raise ValueError before the library is called."""
    with pytest.raises(ValueError):
        call(*tensors())


@pytest.mark.parametrize("call", [
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x, w, residual=x[:3]),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x, w, residual=x.float()),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x, w, total=x),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm(x, w, out=x.float()),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm_grad(x[:2], x, w),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm_grad(x, x, w, d_weight=w[:2]),
    lambda x, w, c, s, i, r, rows, cw: ops.rms_norm_grad(x, x, w, d_total=x.float()),
    lambda x, w, c, s, i, r, rows, cw: ops.route(i, 0),
    lambda x, w, c, s, i, r, rows, cw: ops.route(i, 1025),
    lambda x, w, c, s, i, r, rows, cw: ops.dispatch(x, r, out=rows[:4]),
    lambda x, w, c, s, i, r, rows, cw: ops.combine(rows, r, residual=x.float()),
    lambda x, w, c, s, i, r, rows, cw: ops.combine_grad(x[:2], rows, r, cw),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s, x_scale=torch.ones(4, 1)),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x.to(torch.float8_e4m3fn), c, s),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x.to(torch.float8_e4m3fn), c, s, x_scale=torch.ones(4, 2)),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s, bias=torch.ones(64)),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s, bias=torch.ones(32, dtype=torch.bfloat16)),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s, residual=x),
    lambda x, w, c, s, i, r, rows, cw: ops.linear(x, c, s, out=x),
    lambda x, w, c, s, i, r, rows, cw: ops.linear_grad(x[:, :32], x, c, s, need_dx=False, need_weight=False),
    lambda x, w, c, s, i, r, rows, cw: ops.linear_grad(x[:, :32], x, c, s, d_weight=torch.zeros(64, 16)),
])
def test_tensors_that_do_not_fit_the_others(call, monkeypatch):
    """The same beyond the check for a GPU."""
    monkeypatch.setattr(ops, "_begin", lambda dev, stream: (1, None))
    monkeypatch.setattr(ops, "_scratch", lambda shape, dtype, dev, other: torch.empty(shape, dtype=dtype))
    for name in [n for n in dir(F) if n.startswith("fp8z1_") and not n.endswith(("sizes", "workspace", "dims"))]:
        monkeypatch.setattr(F, name, lambda *a: pytest.fail("the library was called"))
    with pytest.raises(ValueError):
        call(*tensors())


def everything():
    """Each operator once; returns its outputs."""
    x, w, codes, scale, ids, r, rows, cw = tensors()
    out = [*ops.rms_norm(x, w, residual=x), *ops.rms_norm_fp8(x, w, residual=x), *ops.rms_norm_grad(x, x, w), *ops.route(ids, 8),
           ops.dispatch(x, r), ops.combine(rows, r, cw), ops.dispatch_grad(rows, r), *ops.combine_grad(x, rows, r, cw)]
    out += [*ops.linear(x, codes, scale, activation="silu", save=True),
            ops.linear(x.to(torch.float8_e4m3fn), codes, scale, x_scale=torch.ones(4, 1))]
    return out + list(ops.linear_grad(x[:, :32].contiguous(), x, codes, scale, bias=True))


NAMES = ("fp8z1_rms_norm", "fp8z1_rms_norm_grad", "fp8z1_route", "fp8z1_dispatch", "fp8z1_combine", "fp8z1_combine_grad",
         "fp8z1_linear", "fp8z1_linear_grad")


def record(world):  # noqa: F811
    monkeypatch, made, calls = world
    for name in NAMES:
        monkeypatch.setattr(F, name, lambda *a, name=name: calls.append((name, a)))
    return monkeypatch, made, calls


def test_a_call_on_another_stream_takes_that_streams_memory(world):  # noqa: F811
    monkeypatch, made, calls = record(world)
    other = Stream()
    monkeypatch.setattr(ops, "_begin", lambda dev, stream: (other.cuda_stream, other))
    out = everything()
    assert len(calls) == 11 and all(a[-1] == 77 for _, a in calls)
    assert len(made) > len(out)  # workspaces too
    assert all(b.pool is other for b in made), "memory of the current stream's pool, used on another stream"
    assert all("current" in b.users for b in out), "the caller's stream may still read an output that is freed"


def test_a_call_on_the_current_stream_takes_its_memory(world):  # noqa: F811
    monkeypatch, made, calls = record(world)
    monkeypatch.setattr(ops, "_begin", lambda dev, stream: (1, None))
    everything()
    assert len(calls) == 11 and all(b.pool == "current" and not b.users for b in made)
