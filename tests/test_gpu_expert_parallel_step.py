"""The example that runs the expert-parallel operators together around the
exchange: its ranks' routers stay identical, it gives the same results each time,
and its gradients are autograd's of the whole layer on one rank in fp32."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_parallel_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_parallel_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_runs_and_ranks_agree(example):
    sizes = dict(tokens=90, dim=64, ffn=136, experts=12, top=3)
    losses = example.train(ranks=3, steps=4, **sizes)
    assert all(math.isfinite(v) for v in losses)
    assert losses == example.train(ranks=3, steps=4, **sizes)


def test_gradients_are_autograds(example):
    """Normwise.  bf16 roundings (2^-8 of a value) on the way to a gradient: the
    outputs' rows, their weighted sum's gradient, h (dg, du), the expert's own
    result and the sum over a token's copies: 5.  The 8 bits move x, g and u by
    half a step each, at most 2^-6 / 2 of a block's largest value: with blocks of
    32 normal values (largest about 2.1 standard deviations) and errors even over
    the step, 2.1 * 2^-6 / sqrt(12) = 0.0095 of a value's size at most, for each of
    the three, of which a gradient sees two at first order each."""
    layer = example.Layer(ranks=2, tokens=80, dim=64, ffn=96, experts=8, top=2)
    gen = torch.Generator(device="cuda:0").manual_seed(3)
    d_ys = [torch.randn(80, 64, generator=gen, device="cuda:0").to(torch.bfloat16) for _ in layer.ranks]
    balance, z = 0.5, 0.1
    layer.forward()
    logits = [r.logits.clone() for r in layer.ranks]
    layer.backward(d_ys, balance, z)
    router = layer.ranks[0].router.clone().requires_grad_()
    experts = [[w.float().requires_grad_() for w in (r.wg, r.wu, r.wd)] for r in layer.ranks]
    xs = [r.x.float().requires_grad_() for r in layer.ranks]
    load = layer.ranks[0].route[4]
    total = 0.0
    ys = []
    for r, x, zl, dy in zip(layer.ranks, xs, logits, d_ys):
        lg = x @ router.t()
        assert float((lg.detach() - zl).abs().max()) <= 1e-4
        p = torch.softmax(lg, dim=1)
        ids = torch.where(r.route[0] >= 0, r.route[0], 0).long()
        w = p.gather(1, ids)
        w = w / w.sum(dim=1, keepdim=True) * r.valid[:, None]
        y = torch.zeros_like(x)
        for e in range(8):
            wg, wu, wd = (t[e % 4] for t in experts[e // 4])
            out = (torch.nn.functional.silu(x @ wg.t()) * (x @ wu.t())) @ wd.t()
            y = y + out * (w * (ids == e)).sum(dim=1, keepdim=True)
        ys.append(y.detach())
        n = r.valid.sum()
        # each rank's router loss is of its own tokens, the mean over the ranks is what the AllReduce gives
        total = total + (y * dy.float()).sum() + balance * 8 * (load * (p * r.valid[:, None]).sum(dim=0)).sum() / n \
            + z * (torch.logsumexp(lg, dim=1).square() * r.valid).sum() / n
    total.backward()
    near = 5 * 2.0 ** -8 + 2 * 0.0095
    for i, r in enumerate(layer.ranks):
        assert float((r.y.float() - ys[i]).norm()) <= 4 * 2.0 ** -8 * float(ys[i].norm())
        assert bool((r.y[~r.valid] == 0).all()) and bool((r.dx[~r.valid] == 0).all())
        for got, want in ((r.grads[0], experts[i][0].grad), (r.grads[1], experts[i][1].grad), (r.grads[2], experts[i][2].grad), (r.dx, xs[i].grad),
                          (r.d_router, router.grad / 2)):
            assert float((got.float() - want).norm()) <= near * float(want.norm())
