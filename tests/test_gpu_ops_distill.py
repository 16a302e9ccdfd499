"""The distillation loss and its gradient against their definition in 64 bits."""
import math

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


def make(rows, vocab, top, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = (torch.randn(rows, vocab, generator=g, device="cuda") * 2.5).to(dtype)
    ids = torch.randint(0, vocab, (rows, top), generator=g, device="cuda", dtype=torch.int32)  # repeats too
    t = torch.randn(rows, top, generator=g, device="cuda") * 3 + 8
    gone = torch.rand(rows, top, generator=g, device="cuda")
    ids = torch.where(gone < 0.1, torch.full_like(ids, -1), torch.where(gone > 0.95, torch.full_like(ids, vocab), ids))
    t = torch.where((gone > 0.1) & (gone < 0.15), torch.full_like(t, -math.inf), t)
    w = torch.rand(rows, generator=g, device="cuda") * 1024
    return z, ids, t, torch.where(w < 100, torch.zeros_like(w), w)


def check(z, ids, t, w, tau, got_loss, got_d):
    loss, d = R.distill(z, ids, t, tau, w)
    # log total: one rounding of an FP32 exp per term (2 ulp) and of a sum in pieces; a row's loss is a
    # difference of numbers up to about 30 / tau: 1e-5 of their size
    assert ((got_loss.cpu().double() - loss).abs() <= 1e-5 * (loss.abs() + tau * tau * (8 + 30 / tau))).all()
    size = (torch.ones(len(z), dtype=torch.float64) if w is None else w.cpu().double())[:, None] * tau
    q = d / torch.where(size == 0, torch.ones_like(size), size)
    # the gradient: (q - p) to FP32's 1e-5 of q + p, one rounding to its type
    tol = 1e-5 * (q.abs() + 2e-2) * size + (2.0**-8 * d.abs() if got_d.dtype == torch.bfloat16 else 0.0)
    assert ((got_d.cpu().double() - d).abs() <= tol).all()


@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 5, 4), (5, 127, 8), (9, 1000, 16), (2, 4097, 1024),
                                            (17, 32000, 64), (4, 50001, 33), (2, 131072, 128), (1, 300007, 7)])
@pytest.mark.parametrize("dtype,tau", [(torch.bfloat16, 1.0), (torch.float32, 2.0)])
def test_loss_and_gradient(rows, vocab, top, dtype, tau):
    z, ids, t, w = make(rows, vocab, top, dtype, rows * 31 + vocab)
    keep = z.clone()
    loss, d = ops.distill_loss_grad(z, ids, t, temperature=tau, row_weight=w)
    check(keep, ids, t, w, tau, loss, d)
    assert torch.equal(z, keep)
    assert torch.equal(ops.distill_loss(z, ids, t, temperature=tau, row_weight=w), loss)
    again, d2 = ops.distill_loss_grad(z, ids, t, temperature=tau, row_weight=w)
    assert torch.equal(loss, again) and torch.equal(d, d2)
    # in place
    loss3, d3 = ops.distill_loss_grad(z, ids, t, temperature=tau, row_weight=w, out=z)
    assert d3 is z and torch.equal(z, d) and torch.equal(loss3, loss)


@pytest.mark.parametrize("vocab,top,dtype", [(131072, 64, torch.bfloat16), (150001, 1024, torch.bfloat16),
                                             (65537, 5, torch.float32), (57344, 33, torch.float32)])
def test_many_long_rows(vocab, top, dtype):
    """Rows of a CTA each, the first part of which stays in shared memory; the gradient in the logits' place."""
    z, ids, t, w = make(81, vocab, top, dtype, vocab)
    keep = z.clone()
    loss, d = ops.distill_loss_grad(z, ids, t, row_weight=w, out=z)
    check(keep, ids, t, w, 1.0, loss, d)
    again = ops.distill_loss_grad(keep, ids, t, row_weight=w)
    assert torch.equal(loss, again[0]) and torch.equal(d, again[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,lo", [(1000, 0), (1000, 1), (1000, 3), (33333, 5)])
def test_strided_and_unaligned_rows(dtype, vocab, lo):
    z, ids, t, w = make(6, vocab, 9, dtype, vocab + lo)
    wide = torch.full((6, vocab + 29), 3.0, dtype=dtype, device="cuda")
    wide[:, lo:lo + vocab] = z
    out = torch.full((6, vocab + 11), 5.0, dtype=dtype, device="cuda")
    loss, d = ops.distill_loss_grad(wide[:, lo:lo + vocab], ids, t, row_weight=w, out=out[:, lo:lo + vocab])
    check(z, ids, t, w, 1.0, loss, d)
    rest = torch.ones(vocab + 11, dtype=torch.bool, device="cuda")
    rest[lo:lo + vocab] = False
    assert (out[:, rest] == 5).all(), "the gradient reaches outside its rows"


def test_masked_logits_and_empty_rows():
    inf = math.inf
    vocab = 700
    z = torch.randn(8, vocab, device="cuda")
    ids = torch.tensor([[3, 5, 7]] * 8, dtype=torch.int32, device="cuda")
    t = torch.tensor([[2.0, 1.0, 0.0]] * 8, device="cuda")
    w = torch.ones(8, device="cuda")
    z[0, 100:] = -inf                       # masked vocabulary
    z[1, :] = torch.finfo(torch.float32).min  # a mask of the type's lowest value over the whole row
    z[2, 3] = -inf                          # the student gives a listed id nothing
    z[3, :] = -inf                          # nothing left
    w[4] = 0
    z[4, :] = float("nan")                  # weight 0: not read
    ids[5] = torch.tensor([-1, 700, 1 << 30], dtype=torch.int32)  # no entry inside the vocabulary
    t[6] = -inf                             # no entry
    z[7, 9] = float("nan")
    loss, d = ops.distill_loss_grad(z, ids, t, row_weight=w)
    loss, d = loss.cpu(), d.cpu()
    p = torch.softmax(torch.tensor([2.0, 1.0, 0.0], dtype=torch.float64), 0)
    want, wd = R.distill(z[:3].cpu(), ids[:3].cpu(), t[:3].cpu(), 1.0, None)
    assert abs(loss[0] - want[0]) < 1e-4 and (d[0].double() - wd[0]).abs().max() < 1e-6
    assert (d[0, 100:] == 0).all()
    assert abs(loss[1] - ((p * p.log()).sum() + math.log(vocab))) < 1e-4 and (d[1].double() - wd[1]).abs().max() < 1e-6
    assert loss[2] == inf and abs(d[2, 3] + p[0]) < 1e-6
    assert loss[3] == inf and abs(d[3, 3] + p[0]) < 1e-6 and d[3, 8] == 0
    for r in (4, 5, 6):
        assert loss[r] == 0 and (d[r] == 0).all()
    assert loss[7].isnan() and d[7, 500].isnan()


def test_large_and_shifted_logits():
    """Logits of thousands, and a common shift: the running maximum keeps the sum in range."""
    z, ids, t, w = make(4, 5000, 8, torch.float32, 2)
    big = z * 400
    loss, d = ops.distill_loss_grad(big, ids, t, row_weight=w)
    want, wd = R.distill(big, ids, t, 1.0, w)
    assert ((loss.cpu().double() - want).abs() <= 1e-5 * (want.abs() + 5000)).all()
    # a logit of 5000 has an ulp of 2^-11, and the temperature's quotient one rounding: q moves by 2^-11 at most
    assert ((d.cpu().double() - wd).abs() <= 2.0**-10 * w.cpu().double()[:, None]).all()


def test_gradient_against_differences():
    """Differences of the 64-bit loss along random directions."""
    z, ids, t, w = make(5, 300, 6, torch.float32, 77)
    tau = 1.7
    _, d = ops.distill_loss_grad(z, ids, t, temperature=tau, row_weight=w)
    v = torch.randn(z.shape, device="cuda", dtype=torch.float64)
    eps = 1e-4
    up, _ = R.distill(z.double() + eps * v, ids, t, tau, w)
    down, _ = R.distill(z.double() - eps * v, ids, t, tau, w)
    num = ((up - down) / (2 * eps) * w.cpu().double()).sum()
    got = (d.double() * v).sum().cpu()
    # differences: eps^2 of the third derivative; FP32's rounding of the gradient
    assert abs(float(num - got)) <= 1e-5 * float(w.sum()) * tau


def test_many_rows_past_32_bits():
    """Row offsets past 2^32 bytes: the last rows of a large batch."""
    rows, vocab = 40_000, 60_000
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    z[-1] = torch.randn(vocab, device="cuda").bfloat16()
    ids = torch.zeros(rows, 2, dtype=torch.int32, device="cuda")
    ids[:, 1] = 59_999
    t = torch.zeros(rows, 2, device="cuda")
    loss, d = ops.distill_loss_grad(z, ids, t)
    want, wd = R.distill(z[-1:], ids[-1:], t[-1:], 1.0, None)
    assert abs(float(loss[-1].cpu() - want[0])) < 1e-4
    assert ((d[-1].cpu().double() - wd[0]).abs() <= 2.0**-8 * wd[0].abs() + 1e-9).all()
    assert abs(float(loss[0]) - (math.log(vocab) - math.log(2))) < 1e-4


def test_on_another_stream():
    z, ids, t, w = make(6, 9000, 5, torch.float32, 3)
    want = ops.distill_loss_grad(z, ids, t, row_weight=w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        late = z * 1
    loss, d = ops.distill_loss_grad(late, ids, t, row_weight=w, stream=s)
    s.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(d, want[1])
