"""The example that runs the training-step operators with the bucket AllReduce:
its losses fall, its ranks stay identical, and its first step's gradients are
autograd's on the same model in fp32."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distillation_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("distillation_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_losses_fall_and_ranks_agree(example):
    losses = example.train(ranks=3, steps=12, tokens=96, vocab=1001, dim=64, ffn=136)
    assert losses[-1] < 0.8 * losses[0]
    assert losses == example.train(ranks=3, steps=12, tokens=96, vocab=1001, dim=64, ffn=136)


def test_gradients_are_autograds(example):
    """Five bf16 roundings lie between the loss and a gradient (hidden, logits'
    gradient, the block's two, the result's own): 5 * 2^-8 normwise."""
    dev, T, V, D, F, K = "cuda:0", 96, 1001, 64, 136, 16
    r = example.Rank(T, V, D, F, dev)
    g = torch.Generator(device=dev).manual_seed(4)
    ids = torch.randint(0, V, (T,), generator=g, device=dev)
    tids = torch.randint(0, V, (T, K), generator=g, device=dev)
    tlog = torch.randn(T, K, generator=g, device=dev)
    loss = r.step(ids, tids, tlog, 1.5)
    table, wg, wu, wd = (w.float().requires_grad_() for w in r.weights)
    x = table[ids]
    hidden = x + (torch.nn.functional.silu(x @ wg.t()) * (x @ wu.t())) @ wd.t()
    logq = torch.log_softmax(hidden @ table.t() / 1.5, dim=1)
    p = torch.softmax(tlog / 1.5, dim=1)
    want = (p * (p.log() - logq.gather(1, tids))).sum() / T
    want.backward()
    assert abs(loss.item() - want.item()) <= 2 ** -7 * want.item()
    for w, got in zip((table, wg, wu, wd), r.grads):
        assert float((got.float() - w.grad).norm()) <= 5 * 2 ** -8 * float(w.grad.norm())
