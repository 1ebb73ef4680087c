"""ccl_expert_ffn and ccl_expert_ffn_grad with hundreds of calls waiting on the
stream, at widths that no 16-byte row divides and beside whole vectors: every call
gives the bits that it gives alone, and no bounded wait runs out."""
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

from test_gpu_expert_ffn import backward, forward, inputs, saved_of

pytestmark = pytest.mark.gpu


# experts, rows of each, dim, ffn: few rows (the weights as the accumulator's rows) and pairs of CTAs in the forward pass
@pytest.mark.parametrize("experts,rows,D,F", [(48, 10, 766, 218), (48, 70, 766, 218), (48, 70, 768, 224), (20, 130, 301, 97), (3, 400, 1001, 64)])
def test_a_long_queue(experts, rows, D, F):
    sets = []
    for k in range(3):
        counts = [(rows + 7 * e * (k + 1)) % (2 * rows) for e in range(experts)]
        a = inputs(counts, D, F, 70 + k)
        n = a["x"].shape[0]
        saved = saved_of(n, F)
        work = torch.empty(ccl.ccl_plan_expert_ffn_work_bytes(n, experts, D, F, backward=True), dtype=torch.uint8, device="cuda:0")
        sets.append((a, saved, forward(a, saved=saved), backward(a, saved), torch.empty_like(a["x"]), work))
    torch.cuda.synchronize()
    waits = ccl.ccl_gated_ffn_timeouts()
    grads = [{k: torch.empty_like(v) for k, v in s[3].items()} for s in sets]
    for i in range(300):
        a, _, _, _, out, work = sets[i % 3]
        ccl.ccl_expert_ffn(a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], out, work=work)
    for i in range(150):
        (a, saved, _, _, out, work), g = sets[i % 3], grads[i % 3]
        ccl.ccl_expert_ffn(a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], out, saved=saved, work=work)
        ccl.ccl_expert_ffn_grad(a["dy"], a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], saved, g["dx"], g["dwg"], g["dwu"], g["dwd"], work=work)
    torch.cuda.synchronize()
    for (a, _, want, wants, out, _), g in zip(sets, grads):
        assert torch.equal(out, want) and all(torch.equal(g[k], wants[k]) for k in wants)
    assert ccl.ccl_gated_ffn_timeouts() == waits


def test_odd_widths_in_a_graph_and_on_another_stream():
    a = inputs([90, 0, 250, 71], 301, 97, 77)
    n = a["x"].shape[0]
    saved = saved_of(n, 97)
    out = forward(a, saved=saved)
    want = backward(a, saved)
    work = torch.empty(ccl.ccl_plan_expert_ffn_work_bytes(n, 4, 301, 97, backward=True), dtype=torch.uint8, device="cuda:0")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, grads = torch.empty_like(out), {k: torch.zeros_like(v) for k, v in want.items()}

    def step(stream=None):
        ccl.ccl_expert_ffn(a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], got, saved=saved, work=work, stream=stream)
        ccl.ccl_expert_ffn_grad(a["dy"], a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], saved, grads["dx"], grads["dwg"], grads["dwu"],
                                grads["dwd"], work=work, stream=stream)
    step(s)
    s.synchronize()
    assert torch.equal(out, got) and all(torch.equal(want[k], grads[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
        step()
    for t in (got, *grads.values()):
        t.zero_()
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got) and all(torch.equal(want[k], grads[k]) for k in want)
