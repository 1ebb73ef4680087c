"""Data-parallel distillation of a one-block model, every rank simulated on one GPU.

Each rank looks its tokens up (ccl_embedding), runs a gated feed-forward block
with a residual (ccl_gated_ffn), projects onto the tied table, takes the
distillation loss and its gradient in place of the logits (ccl_distill_loss),
and goes back through the block (ccl_gated_ffn_grad) and the table
(ccl_embedding_grad, added to the projection's gradient).  The ranks' gradients
are averaged bucket by bucket (ccl_bucket_allreduce) and every rank takes the
same step, so the ranks' weights stay identical to the bit.

Run: python examples/distillation_step.py [--steps 20] [--ranks 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_allreduce_rank_gb300 as ccl  # noqa: E402

BF16 = torch.bfloat16


class Rank:
    """One rank's weights, gradients and working buffers."""

    def __init__(self, tokens: int, vocab: int, dim: int, ffn: int, device):
        gen = torch.Generator(device=device).manual_seed(0)  # the same weights on every rank

        def weight(rows, cols, std):
            return (torch.randn(rows, cols, generator=gen, device=device) * std).to(BF16)
        self.weights = [weight(vocab, dim, 0.5), weight(ffn, dim, dim ** -0.5), weight(ffn, dim, dim ** -0.5),
                        weight(dim, ffn, ffn ** -0.5)]
        self.grads = [torch.empty_like(w) for w in self.weights]
        self.x, self.y = (torch.empty(tokens, dim, dtype=BF16, device=device) for _ in range(2))
        self.dx = torch.empty_like(self.x)
        self.saved = torch.empty(2, tokens, ffn, device=device)
        self.loss = torch.empty(tokens, device=device)
        self.row_weights = torch.full((tokens,), 1.0 / tokens, device=device)
        need = max(ccl.ccl_plan_gated_ffn_work_bytes(tokens, dim, ffn, backward=True),
                   ccl.ccl_plan_embedding_grad_work_bytes(tokens, vocab, dim))
        self.work = torch.empty(need, dtype=torch.uint8, device=device)

    def step(self, ids, teacher_ids, teacher_logits, temperature: float):
        """The losses of one forward pass; the gradients are left in self.grads."""
        table, wg, wu, wd = self.weights
        d_table, dwg, dwu, dwd = self.grads
        ccl.ccl_embedding(table, ids, self.x)
        ccl.ccl_gated_ffn(self.x, wg, wu, wd, self.y, saved=self.saved, work=self.work)
        hidden = self.x + self.y
        logits = hidden @ table.t()
        ccl.ccl_distill_loss(logits, teacher_ids, teacher_logits, self.loss, grad=logits, weights=self.row_weights,
                             temperature=temperature)
        torch.mm(logits.t(), hidden, out=d_table)
        d_hidden = logits @ table
        ccl.ccl_gated_ffn_grad(d_hidden, self.x, wg, wu, wd, self.saved, self.dx, dwg, dwu, dwd, work=self.work)
        ccl.ccl_embedding_grad(self.dx.add_(d_hidden), ids, d_table, accumulate=True, work=self.work)
        return self.loss.sum()


def train(ranks: int = 4, steps: int = 20, tokens: int = 256, vocab: int = 4000, dim: int = 256, ffn: int = 704, top: int = 16,
          temperature: float = 1.0, rate: float = 0.5, device="cuda:0"):
    """The mean loss of every step; raises if the ranks' weights ever differ,
    or if a kernel gave up waiting (its results are then NaN)."""
    torch.cuda.set_device(device)
    world = [Rank(tokens, vocab, dim, ffn, device) for _ in range(ranks)]
    gen = torch.Generator(device=device).manual_seed(1)
    data = []
    for _ in world:  # each rank its own tokens, with the teacher's top logits for them
        ids = torch.randint(0, vocab, (tokens,), generator=gen, device=device)
        ids[::17] = -1  # padding
        teacher_ids = (ids[:, None] * 7 + torch.arange(top, device=device) * 13 + 1) % vocab
        teacher_ids[ids < 0] = -1  # padding has no teacher
        data.append((ids, teacher_ids, torch.linspace(4, 0, top, device=device).expand(tokens, top).contiguous()))
    mismatches = torch.zeros(1, dtype=torch.int64, device=device)
    losses = []
    for _ in range(steps):
        losses.append(torch.stack([r.step(*d, temperature) for r, d in zip(world, data)]).mean())
        ccl.ccl_bucket_allreduce([r.grads for r in world], op="avg")
        for r in world:
            for w, g in zip(r.weights, r.grads):
                w.sub_(g, alpha=rate)
        for k in range(4):
            ccl.ccl_check_identical([r.weights[k] for r in world], mismatches)
    if ccl.ccl_gated_ffn_timeouts():
        raise RuntimeError("a feed-forward kernel gave up waiting %d times" % ccl.ccl_gated_ffn_timeouts())
    if mismatches.item():
        raise RuntimeError("%d weights differ between ranks" % mismatches.item())
    return [v.item() for v in losses]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--ranks", type=int, default=4)
    args = ap.parse_args()
    losses = train(ranks=args.ranks, steps=args.steps)
    for i, v in enumerate(losses):
        print("step %d loss %.4f" % (i, v))


if __name__ == "__main__":
    main()
