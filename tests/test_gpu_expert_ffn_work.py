"""ccl_expert_ffn in work buffers that were planned for other batches: the sums over K
are cut into the parts that fit, the results keep their bounds, bytes behind the
buffer are not written, and a buffer of the call's own plan or a larger one gives the
same bits."""
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

from test_gpu_expert_ffn import check_forward, forward, inputs, saved_of

pytestmark = pytest.mark.gpu
GUARD = 4096


def in_buffer(a, F, nbytes):
    saved = saved_of(a["x"].shape[0], F)
    work = torch.full((nbytes + GUARD,), 171, dtype=torch.uint8, device="cuda:0")
    out = forward(a, saved=saved, work=work[:nbytes])
    check_forward(a, out, "silu", saved)
    assert bool((work[nbytes:] == 171).all())
    return out


# few rows: one expert, some without rows, odd widths whose copies are in the buffer too
@pytest.mark.parametrize("counts,D,F", [([1], 2048, 1024), ([40], 1024, 2048), ([3, 0, 20, 0, 1], 1024, 776), ([30, 33], 1001, 1333), ([64], 512, 4096)])
def test_a_buffer_planned_for_a_larger_batch(counts, D, F):
    n, e = sum(counts), len(counts)
    a = inputs(counts, D, F, 31)
    plan = lambda rows, **kw: ccl.ccl_plan_expert_ffn_work_bytes(rows, e, D, F, **kw)  # noqa: E731
    want = forward(a)
    assert torch.equal(in_buffer(a, F, plan(n)), want)
    sizes = {plan(r) for r in (n, n + 1, 2 * n, 64 * e, 64 * e + 1, 100 * e)} | {plan(64 * e, backward=True), plan(64 * e + 1, backward=True)}
    assert min(sizes) < plan(n) or n == 1  # there is a smaller one
    for nbytes in sorted(sizes):
        out = in_buffer(a, F, nbytes)
        if nbytes >= plan(n):
            assert torch.equal(out, want)


def test_every_number_of_parts():
    counts, D, F = [17, 30], 1024, 768
    a = inputs(counts, D, F, 32)
    least, most = 47 * F * 2, ccl.ccl_plan_expert_ffn_work_bytes(47, 2, D, F)
    for k in range(9):
        nbytes = least + (most - least) * k // 8
        in_buffer(a, F, nbytes)
    with pytest.raises(ccl.CclError, match="INVALID_ARG"):
        in_buffer(a, F, least - 1)
