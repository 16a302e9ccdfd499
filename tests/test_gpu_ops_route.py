"""Tokens sorted by expert and back, with the gradients, against their definition in 64 bits."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _more as M
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

BF16, F32 = torch.bfloat16, torch.float32


def pick(tokens, top, experts, seed, none=0.0, kind=torch.int32):
    g = M.gen(seed)
    ids = torch.randint(experts, (tokens, top), generator=g, device="cuda")
    ids = torch.where(torch.rand(tokens, top, generator=g, device="cuda") < none, torch.full_like(ids, -1), ids)
    return ids.to(kind)


CHOICES = [(1, 1, 1), (1, 8, 32), (5, 3, 2), (31, 1, 7), (61, 8, 32), (33, 4, 1024), (1000, 2, 17), (4097, 2, 256), (513, 64, 1000),
           (20000, 8, 128), (100_000, 8, 64), (3, 2, 1)]


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("none", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("tokens,top,experts", CHOICES)
def test_sort(tokens, top, experts, none, kind):
    ids = pick(tokens, top, experts, tokens + top, none, kind)
    r = ops.route(ids, experts)
    offsets, place = M.route(ids, experts)
    assert torch.equal(r.offsets.cpu(), offsets) and torch.equal(r.place.cpu(), place)


def test_sort_of_one_expert_and_odd_ids():
    """All choices the same; ids outside the range in either direction; a token that chooses an expert twice."""
    for n in (1, 64, 9000):
        r = ops.route(torch.full((n, 3), 4, device="cuda"), 6)
        assert torch.equal(r.place.reshape(-1).cpu(), torch.arange(3 * n, dtype=torch.int32))
        assert r.offsets.tolist() == [0] * 5 + [3 * n, 3 * n]
    ids = torch.tensor([[-1, 5], [2**40, 0], [-(2**40), 2**32 + 1], [1, 1]], device="cuda")
    r = ops.route(ids, 5)
    assert r.place.tolist() == [[-1, -1], [-1, 0], [-1, -1], [1, 2]] and r.offsets.tolist() == [0, 1, 3, 3, 3, 3]
    r = ops.route(torch.tensor([3, 0, 3], device="cuda"), 4)
    assert r.place.tolist() == [[1], [0], [2]]


def test_no_tokens():
    r = ops.route(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 3)
    assert r.offsets.tolist() == [0, 0, 0, 0] and r.place.shape == (0, 4)
    x = torch.zeros(0, 16, device="cuda")
    rows = ops.dispatch(x, r)
    assert rows.shape == (0, 16) and ops.combine(rows, r).shape == (0, 16)
    d, dw = ops.combine_grad(x, rows, r, torch.zeros(0, 4, device="cuda"))
    assert d.shape == (0, 16) and dw.shape == (0, 4)


def make(tokens, top, experts, dim, dtype, seed, none):
    g = M.gen(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    r = ops.route(pick(tokens, top, experts, seed, none), experts)
    w = torch.rand(tokens, top, generator=g, device="cuda") - 0.3
    return r, w, n(tokens, dim), n(tokens * top, dim), n(tokens, dim), n(tokens, dim)


ROWS = [(1, 1, 1, 1, 0.0), (1, 8, 32, 7168, 0.0), (7, 3, 4, 5, 0.4), (61, 8, 32, 264, 0.0), (100, 2, 9, 1001, 0.2), (300, 17, 40, 130, 0.1),
        (12, 64, 80, 24, 0.5), (2000, 4, 16, 2056, 0.0), (50, 6, 8, 512, 1.0), (9, 9, 3, 16400, 0.1)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,top,experts,dim,none", ROWS)
def test_rows(tokens, top, experts, dim, none, dtype):
    r, w, x, rows, res, dy = make(tokens, top, experts, dim, dtype, tokens + dim, none)
    run(r, w, x, rows, res, dy, dtype)


def run(r, w, x, rows, res, dy, dtype, outs=(None, None, None, None)):
    tokens, top = r.place.shape
    place, last = r.place.long(), int(r.offsets[-1])
    there = place >= 0
    token = torch.arange(tokens, device="cuda")[:, None].expand_as(place)[there]
    at = place[there]
    # gathered rows, bit for bit
    got = ops.dispatch(x, r, out=outs[0])
    want = torch.zeros_like(got)
    want[at] = x[token]
    assert torch.equal(got, want) and not got[last:].any()
    # weighted sums: one rounding, and top FP32 additions relative to the terms
    half, chain = M.half_step(dtype) * 1.01, 2.0**-24 * (top + 2)
    for weight, add in ((w, res), (w, None), (None, None), (None, res)):
        if weight is None:
            y = ops.dispatch_grad(rows, r, add=add, out=outs[1])
        else:
            y = ops.combine(rows, r, weight, residual=add, out=outs[1])
        terms = rows.double()[place.clamp(min=0)] * there[:, :, None] * (1.0 if weight is None else weight.double()[:, :, None])
        want, mag = terms.sum(1), terms.abs().sum(1)
        if add is not None:
            want, mag = want + add.double(), mag + add.double().abs()
        assert ((y.double() - want).abs() <= half * want.abs() + chain * mag + 1e-37).all()
    # gradients
    d_rows, d_w = ops.combine_grad(dy, rows, r, w, out=outs[2])
    want = torch.zeros(rows.shape, dtype=torch.float64, device="cuda")
    want[at] = dy.double()[token] * w.double()[there][:, None]
    assert ((d_rows.double() - want).abs() <= (half + 2.0**-24) * want.abs()).all() and not d_rows[last:].any()
    dots = dy.double()[:, None] * rows.double()[place.clamp(min=0)] * there[:, :, None]
    # FP32 sums of dim terms by up to 256 threads: 2^-24 for each addition in a row
    chain = 2.0**-24 * (dy.shape[1] / 32 + 32)
    assert ((d_w.double() - dots.sum(2)).abs() <= chain * dots.abs().sum(2) + 1e-37).all()
    assert not d_w[~there].any()
    again = ops.combine_grad(dy, rows, r, w)
    assert torch.equal(again[0], d_rows) and torch.equal(again[1], d_w)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,pad,at", [(64, 8, 0), (64, 1, 0), (64, 0, 1), (66, 2, 2), (65, 3, 1), (256, 24, 8)])
def test_strides_and_offsets(dim, pad, at, dtype):
    r, w, x, rows, res, dy = make(40, 3, 5, dim, dtype, dim + pad, 0.2)
    s = [M.strided(t, pad, at) for t in (x, rows, res, dy)]
    outs = [M.strided(torch.zeros_like(t), pad, at) for t in (rows, x, rows)]
    run(r, w, *s, dtype, outs=outs)
    if pad:
        for o in outs:
            assert o.as_strided((o.shape[0] - 1, pad), (dim + pad, 1), o.storage_offset() + dim).isnan().all()


def test_result_over_the_residual():
    r, w, x, rows, res, _ = make(77, 4, 6, 520, BF16, 9, 0.1)
    want = ops.combine(rows, r, w, residual=res)
    got = ops.combine(rows, r, w, residual=res, out=res)
    assert got is res and torch.equal(got, want)


def test_infinities_stay_in_their_tokens():
    """A weight of 0 and a dropped choice: infinities of other rows, or of rows behind the last, are not read."""
    r, w, x, rows, res, dy = make(64, 2, 4, 96, F32, 4, 0.3)
    last = int(r.offsets[-1])
    rows[last:] = float("nan")
    bad = int(r.place.max())
    rows[bad] = float("inf")
    y = ops.combine(rows, r, w, residual=res)
    _, dw = ops.combine_grad(dy, rows, r, w)
    hit = (r.place == bad).any(1)
    assert y[~hit].isfinite().all() and not y[hit].isfinite().any()
    assert dw[r.place != bad].isfinite().all()


def test_more_than_32_bits_of_elements():
    tokens, top, dim = 80_000, 8, 7168  # 4.6e9 elements of rows
    g = M.gen(3)
    ids = torch.randint(32, (tokens, top), generator=g, device="cuda", dtype=torch.int32)
    r = ops.route(ids, 32)
    x = torch.randn(tokens, dim, generator=g, device="cuda", dtype=BF16)
    rows = ops.dispatch(x, r)
    for t in (0, 1, tokens // 2, tokens - 1):
        assert all(torch.equal(rows[p], x[t]) for p in r.place[t].tolist())
    y = ops.combine(rows, r, torch.full((tokens, top), 0.125, device="cuda"))
    assert torch.equal(y, x)  # eight equal rows by an eighth each: every FP32 sum is exact
    d, dw = ops.combine_grad(x, rows, r, torch.ones(tokens, top, device="cuda"))
    assert torch.equal(d, rows)
    norm = x[-5:].double().square().sum(1)[:, None]
    assert ((dw[-5:].double() - norm).abs() <= 2.0**-16 * norm).all()
