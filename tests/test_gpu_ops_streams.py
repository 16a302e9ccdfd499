"""Calls on another stream beside work of the current one: neither may touch the other's memory."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]

LONG = 20_000_000  # clocks: about 10 ms, far longer than the calls


def cases():
    g = torch.Generator(device="cuda").manual_seed(5)
    table, ts = R.fp8_weight(g, 700, 256)
    ids = torch.randint(700, (900,), generator=g, device="cuda")
    gu, gus = R.fp8_weight(g, 2, 256, 512)
    dn, dns = R.fp8_weight(g, 2, 256, 256)
    x = torch.randn(900, 256, generator=g, device="cuda").bfloat16()
    dy = torch.randn(900, 256, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, 400, 900], dtype=torch.int32, device="cuda")
    z = torch.randn(300, 5000, generator=g, device="cuda")
    t_ids = torch.randint(5000, (300, 8), generator=g, device="cuda", dtype=torch.int32)
    t = torch.randn(300, 8, generator=g, device="cuda")

    def ffn(stream):
        y, saved = ops.ffn_forward(x, gu, gus, dn, dns, offsets=off, save=True, stream=stream)
        return (y,) + ops.ffn_backward(dy, x, saved, gu, gus, dn, dns, offsets=off, stream=stream)

    return {
        "embed": lambda stream: (ops.embed(ids, table, ts, stream=stream),),
        "embed_grad": lambda stream: (ops.embed_grad(ids, x, 700, stream=stream),),
        "ffn": ffn,
        "distill": lambda stream: ops.distill_loss_grad(z, t_ids, t, stream=stream),
    }


@pytest.mark.parametrize("name", ["embed", "embed_grad", "ffn", "distill"])
def test_beside_the_same_call_on_the_current_stream(name):
    """The current stream's call waits behind a long kernel while its freed workspace lies in the pool."""
    call = cases()[name]
    want = call(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(LONG)
    first = call(None)
    second = call(s)
    third = call(None)
    torch.cuda.synchronize()
    for got in (first, second, third):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["embed", "embed_grad", "ffn", "distill"])
def test_beside_a_read_of_memory_that_is_freed(name):
    """Blocks of the sizes that the call allocates, still to be read by the current stream, are not written."""
    call = cases()[name]
    sizes = [t.numel() * t.element_size() for t in call(None)] + [1 << k for k in range(12, 25)]
    s = torch.cuda.Stream()
    call(s)
    torch.cuda.synchronize()
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    kept = [torch.empty_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    for k, b in zip(kept, blocks):
        k.copy_(b)
    del blocks, b
    call(s)
    torch.cuda.synchronize()
    assert all((k == 7).all() for k in kept)


def test_clusters_that_start_one_by_one():
    """A row over several CTAs while other kernels hold most of the SMs: no CTA writes to one that has not started."""
    g = torch.Generator(device="cuda").manual_seed(8)
    z = torch.randn(5, 131_072, generator=g, device="cuda")
    ids = torch.randint(131_072, (5, 16), generator=g, device="cuda", dtype=torch.int32)
    t = torch.randn(5, 16, generator=g, device="cuda")
    want = ops.distill_loss_grad(z, ids, t)
    a = torch.randn(2048, 2048, generator=g, device="cuda").bfloat16()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(100):
        with torch.cuda.stream(s):
            a @ a
        got.append(ops.distill_loss_grad(z, ids, t))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for pair in got for x, y in zip(pair, want))
