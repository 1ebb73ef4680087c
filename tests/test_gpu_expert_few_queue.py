"""ccl_expert_ffn for few rows an expert, whole vectors: the second product's kernel
asks for its weights and reads the offsets while the launch before it still runs.
Short queues of small calls whose offsets, rows and weights are written by the
launches right before each: every call gives the bits that it gives alone."""
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

from test_gpu_expert_ffn import inputs

pytestmark = pytest.mark.gpu
DEV, I32 = "cuda:0", torch.int32
CALLS = 24


# one launch a product, sums cut along K with a join between the products, several tiles of an expert
@pytest.mark.parametrize("tokens,experts,top,D,F", [(10, 8, 2, 256, 264), (4, 4, 2, 1024, 2048), (60, 4, 2, 512, 136), (1, 8, 2, 64, 4096)])
def test_each_call_reads_what_was_written_right_before_it(tokens, experts, top, D, F):
    n = tokens * top
    gen = torch.Generator(device=DEV).manual_seed(tokens + D)
    sets = [inputs([0] * experts, D, F, 50 + k, behind=n) for k in range(3)]
    ids = [torch.rand(tokens, experts, generator=gen, device=DEV).argsort(dim=1)[:, :top].to(I32).contiguous() for _ in range(5)]
    x = [torch.randn(tokens, D, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(4)]
    work = torch.empty(ccl.ccl_plan_expert_ffn_work_bytes(n, experts, D, F), dtype=torch.uint8, device=DEV)
    offsets, place = torch.zeros(experts + 1, device=DEV, dtype=I32), torch.zeros(tokens, top, device=DEV, dtype=I32)
    rows, w = torch.zeros(n, D, device=DEV, dtype=torch.bfloat16), [sets[0][k].clone() for k in ("wg", "wu", "wd")]

    def call(i, out, swap):
        if swap:
            for t, k in zip(w, ("wg", "wu", "wd")):
                t.copy_(sets[i % 3][k])
        ccl.ccl_expert_order(ids[i % 5], offsets, place)
        ccl.ccl_dispatch(x[i % 4], place, rows)
        ccl.ccl_expert_ffn(rows, offsets, *w, out, work=work)
    for swap in (True, False):
        alone, queued = ([torch.full((n, D), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(CALLS)] for _ in range(2))
        for i in range(CALLS):
            call(i, alone[i], swap)
            torch.cuda.synchronize()
        work.fill_(255)
        rows.zero_(), offsets.zero_()
        for i in range(CALLS):
            call(i, queued[i], swap)
        torch.cuda.synchronize()
        for i in range(CALLS):
            assert torch.equal(alone[i], queued[i]) and bool(torch.isfinite(alone[i]).all()), (swap, i)
        assert any(not torch.equal(alone[0], o) for o in alone[1:])
    assert ccl.ccl_gated_ffn_timeouts() == 0


def test_in_a_graph():
    """The same as nodes of a graph, replayed on changed offsets."""
    tokens, experts, top, D, F = 12, 8, 2, 512, 1024
    n = tokens * top
    a = inputs([0] * experts, D, F, 60, behind=n)
    ids = torch.zeros(tokens, top, device=DEV, dtype=I32)
    offsets, place = torch.zeros(experts + 1, device=DEV, dtype=I32), torch.zeros(tokens, top, device=DEV, dtype=I32)
    work = torch.empty(ccl.ccl_plan_expert_ffn_work_bytes(n, experts, D, F), dtype=torch.uint8, device=DEV)
    outs = [torch.empty(n, D, dtype=torch.bfloat16, device=DEV) for _ in range(3)]

    def step(out):
        ccl.ccl_expert_order(ids, offsets, place, work=torch.empty(0, dtype=torch.uint8, device=DEV))
        ccl.ccl_expert_ffn(a["x"], offsets, a["wg"], a["wu"], a["wd"], out, work=work)
    step(outs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(outs[1])
        step(outs[2])
    gen = torch.Generator(device=DEV).manual_seed(1)
    for _ in range(4):
        ids.copy_(torch.rand(tokens, experts, generator=gen, device=DEV).argsort(dim=1)[:, :top])
        g.replay()
        torch.cuda.synchronize()
        step(outs[0])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
