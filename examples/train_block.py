"""Distilling a pre-norm block of routed experts on FP8 weights: norm, routing and matrix products around the feed-forward block.

    python examples/train_block.py [steps]

The student is an embedding table, whose transpose gives the logits too, and one block: a norm, a
router that sends each token to its two likeliest experts, gated feed-forward experts whose rows
are joined with the router's weights and added to the stream, and a last norm.  A step is

    embed -> rms_norm -> linear (router) -> route -> dispatch -> ffn_forward -> combine
          -> rms_norm -> linear (logits) -> distill_loss_grad

and back through each one's gradient, then ``ShardOptimizer.step``.  The norms' weights stay FP32
and are torch.optim.Adam's.  Serving takes the last norm's rows in 8 bits.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from blockwise_fp8_zero_fold_gb300 import ops  # noqa: E402
from blockwise_fp8_zero_fold_gb300.optimizer import ShardOptimizer  # noqa: E402
from examples.distill_experts import teacher  # noqa: E402

F32, TOP = torch.float32, 2


class Student:
    def __init__(self, vocab=1000, hidden=256, inner=256, experts=16, seed=0, lr=3e-3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.experts, self.alpha = vocab, experts, hidden**0.5
        shapes = [(1, vocab, hidden), (1, hidden, experts), (experts, hidden, 2 * inner), (experts, inner, hidden)]
        fan_in = [hidden, hidden, hidden, inner]
        self.opt = ShardOptimizer(shapes, lr=lr, weight_decay=0.0)
        self.opt.init_state([torch.randn(s, generator=g, device="cuda") * n**-0.5 for s, n in zip(shapes, fan_in)])
        self.codes = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in shapes]
        self.grads = [torch.zeros(s, dtype=F32, device="cuda") for s in shapes]
        self.opt.step(self.grads, self.codes)  # no gradients yet: writes the FP8 weights and their scales
        self.scales = self.opt.scale_views()
        self.norms = torch.ones(2, hidden, device="cuda")
        self.norms_opt = torch.optim.Adam([self.norms], lr=lr)

    def weight(self, i):
        """An FP8 weight without experts: codes and scales."""
        return self.codes[i][0], self.scales[i][0]

    def experts_weights(self):
        return self.codes[2], self.scales[2], self.codes[3], self.scales[3]

    def router(self, h):
        """Each token's experts and their weights: softmax over its likeliest."""
        z = ops.linear(h, *self.weight(1), dtype=F32)
        best = z.topk(TOP, dim=1)
        return best.indices, best.values.softmax(1)

    def forward(self, ids, save=False):
        """The stream before the last norm, and with ``save`` what the gradients need."""
        x = ops.embed(ids, *self.weight(0), alpha=self.alpha)
        h = ops.rms_norm(x, self.norms[0])
        chosen, w = self.router(h)
        r = ops.route(chosen, self.experts)
        rows = ops.dispatch(h, r)
        y = ops.ffn_forward(rows, *self.experts_weights(), offsets=r.offsets, save=save)
        y, kept = y if save else (y, None)
        out = ops.combine(y, r, w, residual=x)
        return (out, (x, h, chosen, w, r, rows, y, kept)) if save else out

    def logits(self, ids):
        """FP32 logits by way of the last norm's 8-bit rows."""
        codes, scale = ops.rms_norm_fp8(self.forward(ids), self.norms[1])
        return ops.linear(codes, *self.weight(0), x_scale=scale, transposed=True, dtype=F32)

    def gradients(self, ids, teacher_ids, teacher_logits):
        """Each token's loss; the gradients, times the loss scale, in ``grads`` and ``norms.grad``."""
        out, (x, h, chosen, w, r, rows, y, kept) = self.forward(ids, save=True)
        last = ops.rms_norm(out, self.norms[1])
        z = ops.linear(last, *self.weight(0), transposed=True, dtype=F32)
        # the optimizer divides its gradients by the loss scale
        scale = torch.full((len(ids),), self.opt.scaler.scale / len(ids), device="cuda")
        loss, dz = ops.distill_loss_grad(z, teacher_ids, teacher_logits, row_weight=scale, out=z)
        d_last, d_table, _ = ops.linear_grad(dz, last, *self.weight(0), transposed=True)
        d_out, d_norm1 = ops.rms_norm_grad(d_last, out, self.norms[1])
        # the experts' rows, their weights, and the router's logits behind those
        d_y, d_w = ops.combine_grad(d_out, y, r, w)
        d_rows, _, _ = ops.ffn_backward(d_y, rows, kept, *self.experts_weights(), offsets=r.offsets, d_gate_up=self.grads[2],
                                        d_down=self.grads[3])
        d_best = w * (d_w - (w * d_w).sum(1, keepdim=True))
        d_z = torch.zeros(len(ids), self.experts, device="cuda").scatter_(1, chosen, d_best)
        d_h, _, _ = ops.linear_grad(d_z, h, *self.weight(1), d_weight=self.grads[1][0])
        d_h = ops.dispatch_grad(d_rows, r, add=d_h)
        # the stream's gradient past the norm is d_out
        d_x, d_norm0 = ops.rms_norm_grad(d_h, x, self.norms[0], d_total=d_out)
        ops.embed_grad(ids, d_x, self.vocab, alpha=self.alpha, out=self.grads[0][0])
        self.grads[0][0].add_(d_table)  # the table is the logits' weight too
        self.norms.grad = torch.stack([d_norm0, d_norm1])
        return loss

    def train(self, ids, teacher_ids, teacher_logits):
        """One step; returns the mean loss (a device tensor) and the step's found_inf."""
        scale = self.opt.scaler.scale
        loss = self.gradients(ids, teacher_ids, teacher_logits)
        skipped = self.opt.step(self.grads, self.codes)
        if not skipped:
            self.norms.grad.div_(scale)
            self.norms_opt.step()
        return loss.mean(), skipped


def main(steps=30, tokens=1500, top=16):
    student = Student()
    t_ids, t_logits = teacher(student.vocab, top)
    g = torch.Generator(device="cuda").manual_seed(2)
    losses = []
    for i in range(steps):
        ids = torch.randint(student.vocab, (tokens,), generator=g, device="cuda")
        loss, skipped = student.train(ids, t_ids[ids], t_logits[ids])
        losses.append(float(loss))
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i}: loss {losses[-1]:.4f}" + (" (skipped)" if skipped else ""))
    # serving: one token at a time
    z = student.logits(torch.tensor([7], device="cuda"))
    print("after token 7 the student answers", int(z.argmax()), "and the teacher", int(t_ids[7, 0]))
    return losses


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
