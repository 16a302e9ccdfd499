"""What the model operators refuse, and the host side of their sizes: no GPU.

Device pointers are stand-ins (host memory): a call that the library refuses touches none of them."""
import ctypes as C

import numpy as np
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import build as fp8build
from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops


@pytest.fixture(scope="module", autouse=True)
def built():
    fp8build.build()
    return F.lib()


_MEM = np.zeros(4096, np.uint8)
P = (_MEM.ctypes.data + 255) & ~255  # 256-byte aligned


def status(name, *args):
    return getattr(F.lib(), name)(*args)


EMBED = dict(vocab=10, dim=32, codes=P, scales=P, ids=P, id_bytes=8, tokens=4, alpha=1.0, out=P, type=F.BF16, ld=32,
             stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(vocab=0), F.EINVAL), (dict(dim=0), F.EINVAL), (dict(tokens=-1), F.EINVAL), (dict(codes=None), F.EINVAL),
    (dict(scales=None), F.EINVAL), (dict(ids=None), F.EINVAL), (dict(out=None), F.EINVAL), (dict(id_bytes=2), F.EINVAL),
    (dict(type=2), F.EINVAL), (dict(ld=31), F.EINVAL), (dict(alpha=float("nan")), F.EINVAL),
    (dict(tokens=(1 << 30) + 1), F.EINVAL), (dict(ids=P + 4), F.EALIGN), (dict(out=P + 1), F.EALIGN),
    (dict(scales=P + 2), F.EALIGN), (dict(tokens=0, ids=None, out=None), F.OK)])
def test_embed_refusals(change, want):
    a = {**EMBED, **change}
    assert status("fp8z1_embed", *a.values()) == want


GRAD = dict(vocab=10, dim=32, ids=P, id_bytes=8, tokens=4, alpha=1.0, dy=P, type=F.BF16, ld=32, out=P, ws=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(vocab=0), F.EINVAL), (dict(dim=-1), F.EINVAL), (dict(dy=None), F.EINVAL), (dict(out=None), F.EINVAL),
    (dict(ws=None), F.EINVAL), (dict(ld=8), F.EINVAL), (dict(type=-1), F.EINVAL), (dict(id_bytes=16), F.EINVAL),
    (dict(alpha=float("inf")), F.EINVAL), (dict(ws=P + 16), F.EALIGN), (dict(out=P + 2), F.EALIGN),
    (dict(dy=P + 1), F.EALIGN)])
def test_embed_grad_refusals(change, want):
    a = {**GRAD, **change}
    assert status("fp8z1_embed_grad", *a.values()) == want


def test_workspace_sizes():
    n = C.c_int64(-7)
    assert status("fp8z1_embed_grad_workspace", 0, 1, 1, C.byref(n)) == F.EINVAL and n.value == -7
    assert status("fp8z1_embed_grad_workspace", 1, 1, 1, None) == F.EINVAL
    assert F.fp8z1_embed_grad_workspace(131072, 4096, 0) >= 0
    small, large = (F.fp8z1_embed_grad_workspace(1000, 64, t) for t in (10, 100000))
    assert small <= large
    a = F.fp8z1_ffn_sizes(F.fp8z1_ffn_dims(100, 256, 128, 2))
    b = F.fp8z1_ffn_sizes(F.fp8z1_ffn_dims(200, 256, 128, 2))
    assert all(0 < i <= j for i, j in zip(a, b))
    assert all(v >= 0 for v in F.fp8z1_ffn_sizes(F.fp8z1_ffn_dims(0, 256, 128, 2)))
    # the largest sizes do not wrap
    assert all(v > 0 for v in F.fp8z1_ffn_sizes(F.fp8z1_ffn_dims(1 << 30, 16384, 65536, 1024)))


@pytest.mark.parametrize("dims", [(-1, 256, 128, 1), (1, 8, 128, 1), (1, 264, 128, 1), (1, 256, 64, 1), (1, 256, 192, 1),
                                  (1, 256, 0, 1), (1, 0, 128, 1), (1, 256, 128, 0), (1, 256, 128, 1025),
                                  ((1 << 30) + 1, 256, 128, 1), (1, 1 << 24, 128, 1)])
def test_ffn_dims_refused(dims):
    with pytest.raises(F.Fp8z1Error) as e:
        F.fp8z1_ffn_sizes(F.fp8z1_ffn_dims(*dims))
    assert e.value.status == F.EINVAL


FFN = dict(dims=(8, 256, 128, 2), x=P, ld_x=256, off=P, gu=P, gus=P, dn=P, dns=P, y=P, ld_y=256, saved=P, ws=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(x=None), F.EINVAL), (dict(off=None), F.EINVAL), (dict(gu=None), F.EINVAL), (dict(gus=None), F.EINVAL),
    (dict(dn=None), F.EINVAL), (dict(dns=None), F.EINVAL), (dict(y=None), F.EINVAL), (dict(ws=None), F.EINVAL),
    (dict(ld_x=248), F.EINVAL), (dict(ld_y=0), F.EINVAL), (dict(ld_x=260), F.EALIGN), (dict(x=P + 8), F.EALIGN),
    (dict(y=P + 2), F.EALIGN), (dict(gu=P + 8), F.EALIGN), (dict(dn=P + 1), F.EALIGN), (dict(gus=P + 1), F.EALIGN),
    (dict(off=P + 2), F.EALIGN), (dict(saved=P + 16), F.EALIGN), (dict(ws=P + 128), F.EALIGN),
    (dict(dims=(8, 250, 128, 2)), F.EINVAL)])
def test_ffn_forward_refusals(change, want):
    a = {**FFN, **change}
    d = F.fp8z1_ffn_dims(*a.pop("dims"))
    assert status("fp8z1_ffn_forward", C.byref(d), *a.values()) == want


def test_ffn_null_dims():
    assert status("fp8z1_ffn_forward", None, *list(FFN.values())[1:]) == F.EINVAL


BACK = dict(dims=(8, 256, 128, 2), dy=P, ld_dy=256, x=P, ld_x=256, off=P, gu=P, gus=P, dn=P, dns=P, saved=P, dx=P,
            ld_dx=256, d_gu=P, d_dn=P, ws=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(dy=None), F.EINVAL), (dict(x=None), F.EINVAL), (dict(saved=None), F.EINVAL), (dict(d_gu=None), F.EINVAL),
    (dict(d_dn=None), F.EINVAL), (dict(ws=None), F.EINVAL), (dict(ld_dy=128), F.EINVAL), (dict(ld_dx=255), F.EINVAL),
    (dict(ld_dx=257), F.EALIGN), (dict(d_gu=P + 4), F.EALIGN), (dict(d_dn=P + 8), F.EALIGN), (dict(dy=P + 4), F.EALIGN),
    (dict(saved=P + 8), F.EALIGN), (dict(off=None), F.EINVAL)])
def test_ffn_backward_refusals(change, want):
    a = {**BACK, **change}
    d = F.fp8z1_ffn_dims(*a.pop("dims"))
    assert status("fp8z1_ffn_backward", C.byref(d), *a.values()) == want


DISTILL = dict(z=P, type=F.F32, ld=64, rows=2, vocab=64, ids=P, t=P, top=4, tau=1.0, w=P, loss=P, d=P, ld_d=64, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(z=None), F.EINVAL), (dict(type=3), F.EINVAL), (dict(ld=63), F.EINVAL), (dict(rows=-1), F.EINVAL),
    (dict(vocab=0), F.EINVAL), (dict(ids=None), F.EINVAL), (dict(t=None), F.EINVAL), (dict(top=0), F.EINVAL),
    (dict(top=1025), F.EINVAL), (dict(tau=0.0), F.EINVAL), (dict(tau=-1.0), F.EINVAL), (dict(tau=float("inf")), F.EINVAL),
    (dict(tau=float("nan")), F.EINVAL), (dict(loss=None), F.EINVAL), (dict(ld_d=8), F.EINVAL),
    (dict(ld_d=80), F.EINVAL), (dict(z=P + 2), F.EALIGN), (dict(d=P + 1026), F.EALIGN), (dict(ids=P + 1), F.EALIGN),
    (dict(w=P + 2), F.EALIGN), (dict(rows=0, z=None, ids=None, t=None, loss=None, d=None), F.OK)])
def test_distill_refusals(change, want):
    a = {**DISTILL, **change}
    assert status("fp8z1_distill", *a.values()) == want


def test_tensors_that_do_not_fit():
    """ops.py's own checks raise ValueError before the library is called."""
    codes, scale = torch.zeros(300, 200, dtype=torch.uint8), torch.ones(3, 2)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (
        lambda: ops.embed(ids, codes, scale[:2]),                       # scales of another grid
        lambda: ops.embed(ids, codes.float(), scale),                   # not codes
        lambda: ops.embed(ids, codes.t(), scale),                       # not row-major
        lambda: ops.embed(ids.float(), codes, scale),                   # not ids
        lambda: ops.embed(ids, codes, scale, dtype=torch.float16),
        lambda: ops.embed(ids, codes, scale),                           # not on a GPU
        lambda: ops.embed_grad(ids, torch.zeros(5, 8), 10),             # other tokens
        lambda: ops.embed_grad(ids, torch.zeros(4, 8, dtype=torch.float16), 10),
        lambda: ops.distill_loss(torch.zeros(2, 5), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)),
    ):
        with pytest.raises(ValueError):
            call()
    gu, gus = torch.zeros(2, 256, 256, dtype=torch.uint8), torch.ones(2, 2, 2)
    dn, dns = torch.zeros(2, 128, 256, dtype=torch.uint8), torch.ones(2, 1, 2)
    x, off = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(gu=gu[:, :128]), dict(dn=dn[:1]), dict(dns=dns[:, :, :1]),
                dict(off=off.long()), dict(off=off[:2]), dict(off=None), dict()):
        a = {**dict(x=x, gu=gu, gus=gus, dn=dn, dns=dns, off=off), **bad}
        with pytest.raises(ValueError):
            ops.ffn_forward(a["x"], a["gu"], a["gus"], a["dn"], a["dns"], offsets=a["off"])
