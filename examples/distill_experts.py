"""Distilling a small mixture of experts on FP8 weights: the model operators and the optimizer step together.

    python examples/distill_experts.py [steps]

The student is an embedding table (its transpose gives the logits too) and one
layer of gated feed-forward experts with a residual connection; tokens go to
experts by their id.  Its weights live as the optimizer writes them, E4M3 codes
with 128x128 block scales.  A step is

    embed -> ffn_forward -> logits -> distill_loss_grad -> ffn_backward -> embed_grad -> ShardOptimizer.step

and the logits, which belong to no operator here, are a plain FP32 product.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from blockwise_fp8_zero_fold_gb300 import ops  # noqa: E402
from blockwise_fp8_zero_fold_gb300.optimizer import ShardOptimizer  # noqa: E402


class Student:
    def __init__(self, vocab=1024, hidden=256, inner=384, experts=4, seed=0, lr=3e-3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.experts = vocab, experts
        self.alpha = hidden**0.5
        shapes = [(1, vocab, hidden), (experts, hidden, 2 * inner), (experts, inner, hidden)]
        self.opt = ShardOptimizer(shapes, lr=lr, weight_decay=0.0)
        self.opt.init_state([torch.randn(s, generator=g, device="cuda") * s[1 if s[0] > 1 else 2]**-0.5 for s in shapes])
        self.codes = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in shapes]
        self.grads = [torch.zeros(s, dtype=torch.float32, device="cuda") for s in shapes]
        self.opt.step(self.grads, self.codes)  # no gradients yet: writes the FP8 weights and their scales
        self.scales = self.opt.scale_views()
        self.every = torch.arange(vocab, device="cuda")

    def experts_weights(self):
        return self.codes[1], self.scales[1], self.codes[2], self.scales[2]

    def sort_by_expert(self, ids):
        """The tokens grouped by expert, and where each expert's run begins."""
        expert = ids % self.experts
        order = expert.argsort(stable=True)
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.bincount(expert, minlength=self.experts).cumsum(0)
        return ids[order], offsets

    def logits(self, ids, offsets, save=False):
        """FP32 logits of tokens grouped by expert; with ``save`` also what the gradients need."""
        x = ops.embed(ids, self.codes[0][0], self.scales[0][0], alpha=self.alpha)
        y = ops.ffn_forward(x, *self.experts_weights(), offsets=offsets, save=save)
        y, saved = y if save else (y, None)
        out = x.float() + y.float()
        table = ops.embed(self.every, self.codes[0][0], self.scales[0][0], dtype=torch.float32)
        z = out @ table.T
        return (z, (x, saved, out, table)) if save else z

    def train(self, ids, teacher_ids, teacher_logits):
        """One step; returns the mean loss (a device tensor) and the step's found_inf."""
        ids, offsets = ids
        z, (x, saved, out, table) = self.logits(ids, offsets, save=True)
        # the optimizer divides its gradients by the loss scale
        weight = torch.full((len(ids),), self.opt.scaler.scale / len(ids), device="cuda")
        loss, dz = ops.distill_loss_grad(z, teacher_ids, teacher_logits, row_weight=weight)
        d_out = dz @ table
        dx, _, _ = ops.ffn_backward(d_out.bfloat16(), x, saved, *self.experts_weights(), offsets=offsets,
                                    d_gate_up=self.grads[1], d_down=self.grads[2])
        ops.embed_grad(ids, d_out + dx.float(), self.vocab, alpha=self.alpha, out=self.grads[0][0])
        self.grads[0][0].addmm_(dz.T, out)  # the table's gradient as the logits' weight
        return loss.mean(), self.opt.step(self.grads, self.codes)


def teacher(vocab, top, seed=1):
    """What an unseen teacher answers to each token: its `top` likeliest next ones."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = (torch.randn(vocab, vocab, generator=g, device="cuda") * 2).topk(top)
    return logits.indices.int(), logits.values


def main(steps=30, tokens=2000, top=16):
    torch.backends.cuda.matmul.allow_tf32 = False
    student = Student()
    t_ids, t_logits = teacher(student.vocab, top)
    g = torch.Generator(device="cuda").manual_seed(2)
    losses = []
    for i in range(steps):
        ids, offsets = student.sort_by_expert(torch.randint(student.vocab, (tokens,), generator=g, device="cuda"))
        loss, skipped = student.train((ids, offsets), t_ids[ids], t_logits[ids])
        losses.append(float(loss))
        if i % 10 == 0 or i == steps - 1:
            print(f"step {i}: loss {losses[-1]:.4f}" + (" (skipped)" if skipped else ""))
    # serving: one token at a time
    ids, offsets = student.sort_by_expert(torch.tensor([7], device="cuda"))
    z = student.logits(ids, offsets)
    print("after token 7 the student answers", int(z.argmax()), "and the teacher", int(t_ids[7, 0]))
    return losses


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
