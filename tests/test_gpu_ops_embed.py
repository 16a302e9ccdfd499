"""Embedding lookup and its gradient against their definitions in 64 bits."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ids_of(g, n, vocab, dtype, none=0.1):
    """Skewed ids, some of them no token (negative, or past the table)."""
    u = torch.rand(n, generator=g, device="cuda")
    ids = (u * u * u * vocab).long().clamp_(max=vocab - 1)
    bad = torch.rand(n, generator=g, device="cuda")
    ids = torch.where(bad < none / 2, torch.full_like(ids, -1), ids)
    return torch.where(bad > 1 - none / 2, torch.full_like(ids, vocab), ids).to(dtype)


@pytest.mark.parametrize("vocab,dim,tokens", [(1, 1, 1), (300, 200, 7), (129, 257, 300), (1000, 1024, 33),
                                              (5000, 1008, 513), (257, 7168, 64), (64, 16, 4099)])
@pytest.mark.parametrize("dtype,id_type", [(torch.bfloat16, torch.int64), (torch.float32, torch.int32)])
def test_lookup(vocab, dim, tokens, dtype, id_type):
    g = gen(vocab + dim)
    codes, scale = R.fp8_weight(g, vocab, dim)
    ids = ids_of(g, tokens, vocab, id_type)
    got = ops.embed(ids, codes, scale, alpha=3.7, dtype=dtype)
    alpha = torch.tensor(3.7, dtype=torch.float32).double()
    w = R.decode(codes, scale)
    there = (ids >= 0) & (ids < vocab)
    want = torch.where(there[:, None], w[ids.long().clamp(0, vocab - 1)] * alpha.cuda(), torch.zeros((), dtype=torch.float64, device="cuda"))
    # two FP32 products (2^-24 each) and one rounding to the output type
    tol = 2.0**-23 + (2.0**-8 if dtype == torch.bfloat16 else 0.0)
    assert ((got.double() - want).abs() <= 1.01 * tol * want.abs()).all()


def test_lookup_every_code_and_shapes():
    """All 256 codes decode as the format says (the two NaN codes too); ids of
    any shape, strided output rows, an unaligned view."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(2, 1)
    scale = torch.tensor([[0.5, 4.0]], device="cuda")
    ids = torch.tensor([[1, 0], [-1, 1]], device="cuda")
    got = ops.embed(ids, codes, scale, dtype=torch.float32)
    want = R.decode(codes, scale)[ids.clamp(min=0)]
    want[1, 0] = 0
    assert got.shape == (2, 2, 256) and torch.equal(torch.nan_to_num(got.double(), 12345.0), torch.nan_to_num(want, 12345.0))
    wide = torch.full((3, 300), 7.0, device="cuda", dtype=torch.bfloat16)
    out = wide[:, 1:257]
    ops.embed(torch.tensor([0, 1, 0], device="cuda"), codes, scale, out=out)
    assert torch.equal(torch.nan_to_num(out.double(), 9.0), torch.nan_to_num(R.decode(codes, scale)[[0, 1, 0]], 9.0).bfloat16().double())
    assert (wide[:, 0] == 7).all() and (wide[:, 257:] == 7).all()


def test_lookup_offsets_past_32_bits():
    """A table of more than 2^32 codes: the last rows are read."""
    vocab, dim = 600_000, 7168
    codes = torch.zeros(vocab, dim, dtype=torch.uint8, device="cuda")
    codes[-1] = 0x38 + (torch.arange(dim, device="cuda") % 8).to(torch.uint8)
    scale = torch.ones(R.blocks(vocab), R.blocks(dim), device="cuda")
    got = ops.embed(torch.tensor([vocab - 1, 0], device="cuda"), codes, scale)
    assert torch.equal(got[0].float(), 1 + (torch.arange(dim, device="cuda") % 8).float() / 8)
    assert not got[1].any()


@pytest.mark.parametrize("vocab,dim,tokens", [(1, 1, 1), (1, 257, 5000), (300, 200, 7), (129, 256, 300), (50, 1024, 4099),
                                              (5000, 1008, 513), (3, 64, 20000), (2000, 7168, 64), (70000, 48, 9000),
                                              (200000, 16, 3001)])
@pytest.mark.parametrize("dtype,id_type", [(torch.bfloat16, torch.int64), (torch.float32, torch.int32)])
def test_gradient(vocab, dim, tokens, dtype, id_type):
    g = gen(vocab * 7 + dim)
    ids = ids_of(g, tokens, vocab, id_type)
    dy = torch.randn(tokens, dim, generator=g, device="cuda").to(dtype)
    got = ops.embed_grad(ids, dy, vocab, alpha=1.5)
    real = (ids >= 0) & (ids < vocab)
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_put_((ids[real].long(),), dy[real].double() * 1.5, accumulate=True)
    mag = torch.zeros_like(want).index_put_((ids[real].long(),), dy[real].double().abs() * 1.5, accumulate=True)
    # an FP32 sum of n terms is within (n - 1) 2^-24 of their magnitudes, the factor one rounding more
    n = torch.zeros(vocab, dtype=torch.float64, device="cuda").index_put_((ids[real].long(),), torch.ones((), dtype=torch.float64, device="cuda"), accumulate=True)
    assert ((got.double() - want).abs() <= (n[:, None] + 1) * 2.0**-24 * mag).all()
    assert torch.equal(got, ops.embed_grad(ids, dy, vocab, alpha=1.5)), "the gradient does not repeat bit for bit"


@pytest.mark.parametrize("vocab,dim,tokens", [(70001, 512, 700), (70001, 512, 1), (30000, 4096, 5000), (9001, 64, 20000), (3, 40, 17000)])
def test_gradient_of_large_tables(vocab, dim, tokens):
    """Tables cleared beside the sums: every row without a token is zero, the others are not touched by it."""
    g = gen(vocab + tokens)
    ids = (torch.rand(tokens, generator=g, device="cuda").pow(3) * (vocab + 1)).long() - 1  # -1 too; common and rare ids
    ids[-1] = vocab - 1
    dy = torch.randn(tokens, dim, generator=g, device="cuda")
    out = torch.full((vocab, dim), 7.0, device="cuda")
    got = ops.embed_grad(ids, dy, vocab, out=out)
    real = ids >= 0
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, ids[real], dy[real].double())
    mag = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, ids[real], dy[real].double().abs())
    n = torch.bincount(ids[real], minlength=vocab)[:, None]
    assert ((got.double() - want).abs() <= (n + 1) * 2.0**-24 * mag).all()
    again = ops.embed_grad(ids, dy, vocab, out=torch.full_like(out, float("nan")))
    assert torch.equal(got, again)


def test_gradient_of_no_tokens_and_strided_rows():
    g = gen(5)
    none = torch.full((40,), -1, device="cuda")
    out = torch.full((30, 24), 9.0, device="cuda")
    ops.embed_grad(none, torch.full((40, 24), float("nan"), device="cuda"), 30, out=out)
    assert not out.any(), "rows without a token are zero, and what no token reads is not read"
    out.fill_(9.0)
    ops.embed_grad(none[:0], torch.zeros(0, 24, device="cuda"), 30, out=out)
    assert not out.any()
    wide = torch.randn(100, 77, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, 30, (100,), generator=g, device="cuda")
    a = ops.embed_grad(ids, wide[:, 3:43], 30)
    assert torch.equal(a, ops.embed_grad(ids, wide[:, 3:43].contiguous(), 30))


def test_gradient_against_differences():
    """d/dw of sum(dy * lookup) by differences of the 64-bit lookup along random directions."""
    g = gen(11)
    vocab, dim, tokens = 37, 50, 200
    ids = ids_of(g, tokens, vocab, torch.int64)
    dy = torch.randn(tokens, dim, generator=g, device="cuda")
    got = ops.embed_grad(ids, dy, vocab, alpha=2.0).double()
    real = (ids >= 0) & (ids < vocab)

    def f(w):
        return (w[ids[real]] * 2.0 * dy[real].double()).sum()

    w, v = (torch.randn(vocab, dim, generator=g, device="cuda", dtype=torch.float64) for _ in range(2))
    assert abs(float((f(w + v) - f(w - v)) / 2 - (got * v).sum())) <= 1e-4


def test_on_another_stream():
    """Enqueued on a side stream behind its inputs' producer there."""
    s = torch.cuda.Stream()
    codes, scale = R.fp8_weight(gen(1), 500, 256)
    want = ops.embed(torch.arange(500, device="cuda"), codes, scale)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        ids = torch.arange(500, device="cuda")
    got = ops.embed(ids, codes, scale, stream=s)
    grad = ops.embed_grad(ids, got, 500, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(grad, want.float())
