"""How many kernels an embedding gradient takes, as the header says: the zero
rows (dense), the sort (in the same launch up to 4096 tokens), the sums, and
the join once the tokens fill more than one run; and the sums of a run that is
as long as a warp is wide."""
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("n,d,accumulate,launches", [
    (1, 64, False, 2), (8, 64, False, 2), (8, 64, True, 2), (9, 64, False, 3), (9, 64, True, 3),
    (9, 700000, False, 2),   # rows so wide that runs are longer: one run, nothing to join
    (33, 700000, False, 3),  # runs of 32
    (4096, 64, False, 3), (4097, 64, False, 4), (4097, 64, True, 3)])
def test_launches_and_sums(n, d, accumulate, launches):
    rows = 5
    gen = torch.Generator(device=DEV).manual_seed(n)
    ids = torch.randint(-1, rows, (n,), generator=gen, device=DEV)
    dy = torch.randint(-8, 9, (n, d), generator=gen, device=DEV).float()  # whole numbers: every sum is exact
    grad = torch.randint(-8, 9, (rows, d), generator=gen, device=DEV).float()
    want = torch.zeros(rows + 1, d, device=DEV, dtype=torch.float64)
    want.index_add_(0, torch.where(ids < 0, rows, ids), dy.double())
    want = (want[:rows] + (grad.double() if accumulate else 0)).float()
    before = ccl.ccl_launch_count()
    ccl.ccl_embedding_grad(dy, ids, grad, accumulate=accumulate)
    assert ccl.ccl_launch_count() - before == launches
    assert torch.equal(grad, want)
