"""Expert-parallel training of one mixture-of-experts layer, every rank simulated on one GPU.

Each rank has its own tokens, the router's weights, and a shard of the experts.  A step
  - routes the tokens (ccl_route) and averages the experts' loads over the ranks (ccl_allreduce),
  - puts the tokens' copies in expert order (ccl_expert_order, ccl_dispatch) and sends them to the experts' ranks
    (ccl_alltoallv), where the rows of all sources are put in expert order once more,
  - runs the experts' feed-forward blocks (ccl_expert_ffn), x, g and u being kept in 8 bits (ccl_act8_pack),
  - sends the rows back and sums them with the router's weights (ccl_combine),
and goes back the same way: ccl_combine_grad, the exchange, ccl_expert_ffn_grad, the exchange, ccl_combine (the gradient
of the dispatch) and ccl_route_grad with the balance and z losses.  The router's gradient is averaged over the ranks
(ccl_allreduce); the experts' gradients are whole where they are, since all their tokens were sent there.

Run: python examples/expert_parallel_step.py [--steps 20] [--ranks 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_allreduce_rank_gb300 as ccl  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


def _act8(rows: int, cols: int, device):
    """Room for rows of `cols` values in 8 bits."""
    width = ccl.ccl_plan_act8_width(cols)
    return torch.empty(rows, width, dtype=torch.int8, device=device), torch.empty(rows, width // 32, dtype=torch.uint8, device=device)


class Rank:
    """One rank's tokens, weights and gradients."""

    def __init__(self, rank: int, ranks: int, tokens: int, dim: int, ffn: int, experts: int, top: int, device):
        local = experts // ranks
        same = torch.Generator(device=device).manual_seed(0)          # the router is the same on every rank
        mine = torch.Generator(device=device).manual_seed(1 + rank)   # the experts are not

        def weight(gen, *shape):
            return (torch.randn(*shape, generator=gen, device=device) * shape[-1] ** -0.5).to(BF16)
        self.router = torch.randn(experts, dim, generator=same, device=device) * dim ** -0.5
        self.wg, self.wu = weight(mine, local, ffn, dim), weight(mine, local, ffn, dim)
        self.wd = weight(mine, local, dim, ffn)
        self.x = torch.randn(tokens, dim, generator=mine, device=device).to(BF16)
        self.target = torch.randn(tokens, dim, generator=mine, device=device).to(BF16)
        self.valid = torch.ones(tokens, dtype=torch.bool, device=device)
        self.valid[::17] = False  # padding
        e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        self.route = [e(tokens, top, dtype=I32), e(tokens, top), e(tokens), e(experts + 1, dtype=I32), e(experts), e(experts), e(2)]
        self.offsets, self.place = e(experts + 1, dtype=I32), e(tokens, top, dtype=I32)
        self.send, self.back, self.d_back = (torch.zeros(tokens * top, dim, dtype=BF16, device=device) for _ in range(3))
        self.y, self.dx = torch.empty_like(self.x), torch.empty_like(self.x)
        self.grads = [torch.empty_like(w) for w in (self.wg, self.wu, self.wd)]


class Layer:
    """The layer on all ranks, with its forward and backward pass."""

    def __init__(self, ranks: int = 4, tokens: int = 256, dim: int = 128, ffn: int = 352, experts: int = 16, top: int = 2, device="cuda:0"):
        torch.cuda.set_device(device)
        self.n, self.dim, self.ffn, self.experts, self.top, self.device = ranks, dim, ffn, experts, top, device
        self.local = experts // ranks
        self.ranks = [Rank(r, ranks, tokens, dim, ffn, experts, top, device) for r in range(ranks)]

    def _exchange(self, send, recv, counts):
        ccl.ccl_alltoallv(send, recv, [[c * self.dim for c in row] for row in counts])

    def forward(self) -> None:
        for r in self.ranks:
            r.logits = r.x.float() @ r.router.t()
            ccl.ccl_route(r.logits, *r.route, valid=r.valid)
            ccl.ccl_expert_order(r.route[0], r.offsets, r.place)
            ccl.ccl_dispatch(r.x, r.place, r.send)
        loads = [r.route[4] for r in self.ranks]
        ccl.ccl_allreduce(loads, op="avg")  # the balance loss looks at all ranks' tokens
        # what goes where: the exchange's counts are host numbers
        offsets = torch.stack([r.offsets for r in self.ranks]).cpu()
        rows = offsets[:, 1:] - offsets[:, :-1]                                  # [source, expert]
        by_rank = rows.view(self.n, self.n, self.local).sum(dim=2).tolist()      # [source, destination]
        self.counts, self.returned = by_rank, [list(c) for c in zip(*by_rank)]
        for j, r in enumerate(self.ranks):
            mine = rows[:, j * self.local:(j + 1) * self.local].reshape(-1)      # (source, expert) blocks as they arrive
            ids = torch.arange(self.local, dtype=I32).repeat(self.n).repeat_interleave(mine).to(self.device)
            total = ids.numel()
            e = lambda: torch.empty(total, self.dim, dtype=BF16, device=self.device)  # noqa: E731
            r.ids2, r.place2 = ids[:, None].contiguous(), torch.empty(total, 1, dtype=I32, device=self.device)
            r.offsets2 = torch.empty(self.local + 1, dtype=I32, device=self.device)
            r.arrived, r.grouped, r.out, r.leaving = e(), e(), e(), e()
            r.x8 = _act8(total, self.dim, self.device)
            saved = _act8(2 * total, self.ffn, self.device)
            r.saved = tuple(t.view(2, total, -1) for t in saved)
            r.work = torch.empty(ccl.ccl_plan_expert_ffn_work_bytes(total, self.local, self.dim, self.ffn, backward=True),
                                 dtype=torch.uint8, device=self.device)
        self._exchange([r.send for r in self.ranks], [r.arrived for r in self.ranks], self.counts)
        for r in self.ranks:
            ccl.ccl_expert_order(r.ids2, r.offsets2, r.place2)
            ccl.ccl_dispatch(r.arrived, r.place2, r.grouped)
            ccl.ccl_act8_pack(r.grouped, *r.x8)  # the rows themselves are not kept
            ccl.ccl_expert_ffn(r.grouped, r.offsets2, r.wg, r.wu, r.wd, r.out, saved=r.saved, work=r.work)
            ccl.ccl_combine(r.out, r.place2, r.leaving)
        self._exchange([r.leaving for r in self.ranks], [r.back for r in self.ranks], self.returned)
        for r in self.ranks:
            ccl.ccl_combine(r.back, r.place, r.y, weights=r.route[1])

    def backward(self, d_ys, balance: float = 1e-2, z: float = 1e-3) -> None:
        """The gradients by the experts' weights (rank.grads), the router's
        weights (rank.d_router, averaged) and the tokens (rank.dx)."""
        for r, dy in zip(self.ranks, d_ys):
            r.d_weights = torch.empty_like(r.route[1])
            ccl.ccl_combine_grad(dy, r.place, rows=r.back, weights=r.route[1], grad_rows=r.d_back, grad_weights=r.d_weights)
        self._exchange([r.d_back for r in self.ranks], [r.arrived for r in self.ranks], self.counts)
        for r in self.ranks:
            ccl.ccl_dispatch(r.arrived, r.place2, r.out)
            ccl.ccl_expert_ffn_grad(r.out, r.x8, r.offsets2, r.wg, r.wu, r.wd, r.saved, r.grouped, *r.grads, work=r.work)
            ccl.ccl_combine(r.grouped, r.place2, r.leaving)
        self._exchange([r.leaving for r in self.ranks], [r.d_back for r in self.ranks], self.returned)
        for r in self.ranks:
            ids, _, lse, counts, load = r.route[:5]
            ccl.ccl_combine(r.d_back, r.place, r.dx)  # the dispatch's gradient
            ccl.ccl_route_grad(r.logits, ids, lse, counts, load, r.d_weights, r.logits, balance=balance, z=z)
            r.d_router = r.logits.t() @ r.x.float()
            r.dx.add_(r.logits @ r.router)
        ccl.ccl_allreduce([r.d_router for r in self.ranks], op="avg")


def train(ranks: int = 4, steps: int = 20, rate: float = 0.5, **sizes):
    """The mean squared error of every step; raises if the routers ever differ,
    or if a kernel gave up waiting (its results are then NaN)."""
    layer = Layer(ranks, **sizes)
    mismatches = torch.zeros(1, dtype=torch.int64, device=layer.device)
    losses = []
    for _ in range(steps):
        layer.forward()
        off = [(r.y.float() - r.target.float()) * r.valid[:, None] for r in layer.ranks]
        losses.append(torch.stack([d.square().mean() for d in off]).mean())
        layer.backward([(d * (2 / d.shape[0])).to(BF16) for d in off])
        for r in layer.ranks:
            r.router.sub_(r.d_router, alpha=rate)
            for w, g in zip((r.wg, r.wu, r.wd), r.grads):
                w.sub_(g, alpha=rate / ranks)
        ccl.ccl_check_identical([r.router for r in layer.ranks], mismatches)
    if ccl.ccl_gated_ffn_timeouts():
        raise RuntimeError("a feed-forward kernel gave up waiting %d times" % ccl.ccl_gated_ffn_timeouts())
    if mismatches.item():
        raise RuntimeError("%d of the routers' weights differ between ranks" % mismatches.item())
    return [v.item() for v in losses]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--ranks", type=int, default=4)
    args = ap.parse_args()
    for i, v in enumerate(train(ranks=args.ranks, steps=args.steps)):
        print("step %d loss %.4f" % (i, v))


if __name__ == "__main__":
    main()
