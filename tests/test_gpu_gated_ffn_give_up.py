"""A wait of the feed-forward block that runs out shows in the data: every
output that needed it is NaN, whatever the buffers held, and the waits are
counted.  The limit of the waits is set from the host to 0, so that the kernels
give up at once and return; nothing hangs.  In a child process, because the
other tests ask for a count of 0."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

CHILD = r"""
import importlib.util, sys
import torch
sys.path.insert(0, %r)
import ring_allreduce_rank_gb300 as ccl

DEV, BF16 = "cuda:0", torch.bfloat16


def buffers(T, D, F, fill):
    full = lambda *s: torch.full(s, fill, dtype=BF16, device=DEV)
    work = full(ccl.ccl_plan_gated_ffn_work_bytes(T, D, F, backward=True) // 2)  # finite wherever it is read as bf16
    return full(T, D), torch.full((2, T, F), fill, device=DEV), [full(T, D), full(F, D), full(F, D), full(D, F)], work


seen = 0
# both kernels, with and without sums cut along K, aligned rows and odd ones, several tiles of a pair
for T, D, F in ((1, 512, 1024), (40, 128, 264), (48, 4096, 1024), (70, 37, 41), (200, 129, 255), (300, 520, 1000), (3000, 256, 1536)):
    gen = torch.Generator(device=DEV).manual_seed(T)
    rand = lambda r, c: (torch.randn(r, c, generator=gen, device=DEV) * c ** -0.5).to(BF16)
    x, wg, wu, wd, dy = rand(T, D), rand(F, D), rand(F, D), rand(D, F), rand(T, D)

    def both(out, saved, grads, work, accumulate=False):
        ccl.ccl_gated_ffn(x, wg, wu, wd, out, saved=saved, work=work)
        kept = saved.clone()
        if accumulate is None:
            saved = good[1]  # what the backward pass reads is sound
        ccl.ccl_gated_ffn_grad(dy, x, wg, wu, wd, saved, *grads, work=work, accumulate=bool(accumulate))
        return [out, kept, *grads]

    good = buffers(T, D, F, 5.0)
    want = both(*good)
    assert ccl.ccl_gated_ffn_timeouts() == seen
    assert all(bool(torch.isfinite(t).all()) for t in want)
    ccl.ccl_set_gated_ffn_wait_limit(0)
    for accumulate in (False, True, None):
        for name, t in zip(("out", "saved", "dx", "dwg", "dwu", "dwd"), both(*buffers(T, D, F, 5.0), accumulate)):
            assert bool(torch.isnan(t).all()), (T, D, F, name, accumulate, int(torch.isnan(t).sum()), t.numel())
    seen = ccl.ccl_gated_ffn_timeouts()
    assert seen > 0
    ccl.ccl_set_gated_ffn_wait_limit(4 * 10 ** 9)
    for a, b in zip(want, both(*buffers(T, D, F, 7.0))):  # the device works on as before
        assert torch.equal(a, b)
    assert ccl.ccl_gated_ffn_timeouts() == seen

# a training loop that asks at its end
spec = importlib.util.spec_from_file_location("distillation_step", %r)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)
try:
    example.train(ranks=2, steps=1, tokens=32, vocab=100, dim=64, ffn=136)
except RuntimeError as e:
    print("raised:", e)
print("give up ok")
""" % (ROOT, os.path.join(ROOT, "examples", "distillation_step.py"))


def test_outputs_of_waits_that_ran_out_are_nan():
    res = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "give up ok" in res.stdout and "raised: a feed-forward kernel gave up waiting" in res.stdout
