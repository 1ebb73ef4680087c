"""A wait of the experts' feed-forward blocks that runs out shows in the data:
every output that needed it is NaN, whatever the buffers held, rows of no expert
are left alone, and the waits are counted.  The limit of the waits is set from the
host to 0, so that the kernels give up at once and return; nothing hangs.  In a
child process, because the other tests ask for a count of 0."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

CHILD = r"""
import sys
import torch
sys.path.insert(0, %r)
import ring_allreduce_rank_gb300 as ccl

DEV, BF16 = "cuda:0", torch.bfloat16
seen = 0
# both kernels of the forward pass, with and without sums cut along K, aligned rows and odd ones, several tiles of a pair, an expert without rows
for counts, D, F in (([2], 512, 1024), ([20, 0, 17], 128, 264), ([30, 9], 37, 41), ([200, 0, 150], 129, 255), ([300, 500], 520, 1000), ([3000], 256, 1536)):
    E, N = len(counts), sum(counts) + 3
    gen = torch.Generator(device=DEV).manual_seed(D)
    rand = lambda *s: (torch.randn(*s, generator=gen, device=DEV) * s[-1] ** -0.5).to(BF16)
    x, wg, wu, wd, dy = rand(N, D), rand(E, F, D), rand(E, F, D), rand(E, D, F), rand(N, D)
    offsets = torch.tensor([0] + counts, device=DEV).cumsum(0).to(torch.int32)
    width = ccl.ccl_plan_act8_width(F)

    def buffers(fill):
        full = lambda *s: torch.full(s, fill, dtype=BF16, device=DEV)
        work = torch.full((ccl.ccl_plan_expert_ffn_work_bytes(N, E, D, F, backward=True) // 2 + 1,), fill, dtype=BF16, device=DEV)
        saved = (torch.ones(2, N, width, dtype=torch.int8, device=DEV), torch.full((2, N, width // 32), 120, dtype=torch.uint8, device=DEV))
        return full(N, D), saved, [full(N, D), full(E, F, D), full(E, F, D), full(E, D, F)], work

    def both(out, saved, grads, work, accumulate=False, kept=None):
        ccl.ccl_expert_ffn(x, offsets, wg, wu, wd, out, saved=saved, work=work)
        ccl.ccl_expert_ffn_grad(dy, x, offsets, wg, wu, wd, kept or saved, *grads, work=work, accumulate=accumulate)
        return [out, *grads]

    good = buffers(5.0)
    want = both(*good)
    assert ccl.ccl_gated_ffn_timeouts() == seen
    assert all(bool(torch.isfinite(t).all()) for t in want)
    ccl.ccl_set_gated_ffn_wait_limit(0)
    rows = N - 3
    for accumulate, kept in ((False, None), (True, None), (False, good[1])):
        b = buffers(5.0)
        out, dx, *dw = both(*b, accumulate, kept)
        for t in (out, dx):
            assert bool(torch.isnan(t[:rows]).all()) and bool((t[rows:] == 5).all()), (counts, D, F, accumulate)
        assert bool((b[1][1][:, :rows] == 255).all()) and bool((b[1][1][:, rows:] == 120).all())
        for g in dw:
            for e, n in enumerate(counts):
                assert bool(torch.isnan(g[e]).all() if n else (g[e] == (5 if accumulate else 0)).all()), (counts, D, F, e, accumulate)
    seen = ccl.ccl_gated_ffn_timeouts()
    assert seen > 0
    ccl.ccl_set_gated_ffn_wait_limit(4 * 10 ** 9)
    for a, b in zip(want, both(*buffers(7.0))):  # the device works on as before
        assert torch.equal(a[:rows] if a.shape[0] == N else a, b[:rows] if b.shape[0] == N else b)
    assert ccl.ccl_gated_ffn_timeouts() == seen
print("give up ok")
""" % ROOT


def test_outputs_of_waits_that_ran_out_are_nan():
    res = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "give up ok" in res.stdout
