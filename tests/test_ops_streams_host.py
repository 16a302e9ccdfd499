"""Where the model operators' memory comes from when a call goes to another stream: no GPU.

torch's allocator orders a block's next life behind its last one on the stream whose pool it belongs to, and on no other.
What a call on another stream allocates has to come from that stream's pool."""
import contextlib

import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import fp8z1 as F
from blockwise_fp8_zero_fold_gb300 import ops


class Stream:
    cuda_stream = 77


class Block:
    """A tensor that says which stream's pool it is from and who else uses it."""

    def __init__(self, shape, pool):
        self.shape, self.pool, self.users = torch.Size(shape if hasattr(shape, "__len__") else (shape,)), pool, []

    def record_stream(self, s):
        self.users.append(s)

    def stride(self):
        return (self.shape[-1], 1)

    def dim(self):
        return len(self.shape)


@pytest.fixture
def world(monkeypatch):
    """Streams, allocations and the library's calls without a GPU."""
    now, made, calls = ["current"], [], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(shape, **_):
        made.append(Block(shape, now[-1]))
        return made[-1]

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[-1])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(ops, "_same_device", lambda dev, *t: None)
    for name in ("fp8z1_embed", "fp8z1_embed_grad", "fp8z1_ffn_forward", "fp8z1_ffn_backward", "fp8z1_distill"):
        monkeypatch.setattr(F, name, lambda *a, name=name: calls.append((name, a)))
    monkeypatch.setattr(F, "fp8z1_embed_grad_workspace", lambda *a: 512)
    monkeypatch.setattr(F, "fp8z1_ffn_sizes", lambda d: (256, 512, 768))
    return monkeypatch, made, calls


def everything():
    """Each operator once; returns its outputs."""
    codes, scale = torch.zeros(300, 256, dtype=torch.uint8), torch.ones(3, 2)
    ids, dy = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 256)
    gu, gus = torch.zeros(2, 256, 256, dtype=torch.uint8), torch.ones(2, 2, 2)
    dn, dns = torch.zeros(2, 128, 256, dtype=torch.uint8), torch.ones(2, 1, 2)
    x, off = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    z, t_ids, t = torch.zeros(2, 9), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    out = [ops.embed(ids, codes, scale), ops.embed_grad(ids, dy, 300)]
    out += ops.ffn_forward(x, gu, gus, dn, dns, offsets=off, save=True)
    out += ops.ffn_backward(x, x, torch.zeros(256, dtype=torch.uint8), gu, gus, dn, dns, offsets=off)
    return out + [ops.distill_loss(z, t_ids, t)] + list(ops.distill_loss_grad(z, t_ids, t))


def test_a_call_on_another_stream_takes_that_streams_memory(world):
    monkeypatch, made, calls = world
    other = Stream()
    monkeypatch.setattr(ops, "_begin", lambda dev, stream: (other.cuda_stream, other))
    out = everything()
    assert len(calls) == 6 and all(a[-1] == 77 for _, a in calls)
    assert len(made) > len(out)  # workspaces too
    assert all(b.pool is other for b in made), "memory of the current stream's pool, used on another stream"
    assert all("current" in b.users for b in out), "the caller's stream may still read an output that is freed"


def test_a_call_on_the_current_stream_takes_its_memory(world):
    monkeypatch, made, calls = world
    monkeypatch.setattr(ops, "_begin", lambda dev, stream: (1, None))
    everything()
    assert len(calls) == 6 and all(b.pool == "current" and not b.users for b in made)
