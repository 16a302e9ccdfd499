"""The operators together, as the example trains with them: a step's gradients, and that training learns."""
import pytest
import torch

from blockwise_fp8_zero_fold_gb300 import ops
from examples import distill_experts as X
from tests import _ops as R
from tests._gpu import lib  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("lib")]


def test_gradients_of_the_whole_step():
    """Against autograd in 64 bits through the decoded weights.  Beside FP32 the step rounds x, h, y, d_out, dx and
    [dg | du] to BF16's 8 bits, 2^-9 of the norm at most each (uniform errors: half that), and their effects add up
    over the chain: 6 * 2^-9 = 1.2 %."""
    s = X.Student(vocab=520, hidden=144, inner=256, experts=3)
    g = torch.Generator(device="cuda").manual_seed(3)
    ids, offsets = s.sort_by_expert(torch.randint(s.vocab, (301,), generator=g, device="cuda"))
    t_ids, t_logits = X.teacher(s.vocab, 9)
    w = [R.decode(c, v).requires_grad_() for c, v in zip(s.codes, s.scales)]
    scale = s.opt.scaler.scale
    loss, found = s.train((ids, offsets), t_ids[ids], t_logits[ids])
    assert found == 0

    x = s.alpha * w[0][0][ids]
    out = []
    for e, (lo, hi) in enumerate(R.runs(offsets, 3, len(ids))):
        gate, up = (x[lo:hi] @ w[1][e]).chunk(2, 1)
        out.append(x[lo:hi] + (torch.nn.functional.silu(gate) * up) @ w[2][e])
    q = (torch.cat(out) @ w[0][0].T).log_softmax(1)
    p = t_logits[ids].double().log_softmax(1)
    want = (p.exp() * (p - q.gather(1, t_ids[ids].long()))).sum(1).mean()
    want.backward()
    assert abs(float(loss) - want.item()) <= 6 * 2.0**-9 * abs(want.item())
    for got, ref in zip(s.grads, w):
        ref = ref.grad * scale
        assert float((got.double() - ref).norm()) <= 6 * 2.0**-9 * float(ref.norm())


def test_training_learns():
    losses = X.main(steps=40, tokens=1000, top=8)
    assert losses[-1] < 0.7 * losses[0]


def test_a_pass_can_be_captured():
    """Forward and backward in a CUDA graph, replayed on new inputs."""
    s = X.Student()
    ids, offsets = s.sort_by_expert(torch.arange(600, device="cuda"))
    w = s.experts_weights()
    x = ops.embed(ids, s.codes[0][0], s.scales[0][0], alpha=s.alpha)
    dy = torch.randn(600, 256, device="cuda").bfloat16()

    def step():
        y, saved = ops.ffn_forward(x, *w, offsets=offsets, save=True)
        few = ops.ffn_forward(x[:3], *(t[:1] for t in w))
        loss, dz = ops.distill_loss_grad(y, t_ids, t_logits)
        return (y, few, loss, dz, ops.embed_grad(ids, y, s.vocab)) + ops.ffn_backward(dy, x, saved, *w, offsets=offsets)

    t_ids = torch.randint(256, (600, 5), device="cuda", dtype=torch.int32)
    t_logits = torch.randn(600, 5, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.mul_(-0.5)
    dy.mul_(3)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
