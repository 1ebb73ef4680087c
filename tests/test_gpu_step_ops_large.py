"""The training-step operators on matrices whose byte offsets pass 32 bits
(5 to 6 GB each): the rows at both ends against small calls on those rows alone,
which the other tests hold to the formulas."""
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def test_embedding_and_its_gradient():
    rows, d, n = 330000, 8200, 600  # 5.4 GB
    gen = torch.Generator(device=DEV).manual_seed(1)
    table = torch.empty(rows, d, dtype=BF16, device=DEV)
    ends = torch.cat([torch.arange(3, device=DEV), torch.arange(rows - 3, rows, device=DEV)])
    table[ends] = torch.randn(6, d, generator=gen, device=DEV).to(BF16)
    ids = ends[torch.randint(0, 6, (n,), generator=gen, device=DEV)]
    out, small = torch.empty(n, d, dtype=BF16, device=DEV), torch.empty(n, d, dtype=BF16, device=DEV)
    at = torch.where(ids < 3, ids, ids - rows + 6)
    ccl.ccl_embedding(table, ids, out, scale=1.5)
    ccl.ccl_embedding(table[ends].contiguous(), at, small, scale=1.5)
    assert torch.equal(out, small)
    for count in (n, 8 * n):  # ranked by counting, and sorted
        dy = torch.randn(count, d, generator=gen, device=DEV).to(BF16)
        which, there = ids.repeat(count // n), at.repeat(count // n)
        grad = torch.empty(6, d, dtype=BF16, device=DEV)
        table.fill_(3.0)
        ccl.ccl_embedding_grad(dy, which, table, scale=1.5)
        ccl.ccl_embedding_grad(dy, there, grad, scale=1.5)
        assert torch.equal(table[ends], grad)
        assert not bool(table[3:rows - 3].any())


@pytest.mark.parametrize("dtype,T,V", [(BF16, 21000, 128003), (torch.float32, 11000, 128003)])
def test_distillation(dtype, T, V):
    gen = torch.Generator(device=DEV).manual_seed(2)
    logits = torch.zeros(T, V, dtype=dtype, device=DEV)
    ends = [0, 1, T - 2, T - 1]
    logits[ends] = torch.randn(4, V, generator=gen, device=DEV).to(dtype)
    small = logits[ends].contiguous()
    ids = torch.randint(0, V, (T, 20), generator=gen, device=DEV)
    teacher = torch.randn(T, 20, generator=gen, device=DEV)
    loss, stats, few = torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV), torch.empty(4, device=DEV)
    kept, grad = torch.empty(4, 2, device=DEV), torch.empty_like(small)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, stats=stats)
    ccl.ccl_distill_loss(small, ids[ends].contiguous(), teacher[ends].contiguous(), few, stats=kept, grad=grad)
    # another number of rows may take other parts of a row: sums in another order
    assert bool(((loss[ends] - few).abs() <= 2.0 ** -16 * (few.abs() + 20)).all())
    assert torch.equal(stats[ends][:, 0], kept[:, 0])
    ccl.ccl_distill_loss(logits, ids, teacher, loss, grad=logits)
    got = logits[ends].double()
    unit = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    assert bool(((got - grad.double()).abs() <= (2.0 ** -14 + 2 * unit) * grad.double().abs() + 1e-9).all())


def test_gated_ffn():
    T, D, F = 90000, 64, 16384  # g and u 5.9 GB each, h 2.9 GB
    gen = torch.Generator(device=DEV).manual_seed(3)
    rand = lambda r, c, s: (torch.randn(r, c, generator=gen, device=DEV) * s).to(BF16)  # noqa: E731
    x, wg, wu, wd, dy = rand(T, D, 1.0), rand(F, D, D ** -0.5), rand(F, D, D ** -0.5), rand(D, F, F ** -0.5), rand(T, D, 0.1)
    ends = torch.cat([torch.arange(256, device=DEV), torch.arange(T - 256, T, device=DEV)])
    out, dx, saved = torch.empty_like(x), torch.empty_like(x), torch.empty(2, T, F, device=DEV)
    ccl.ccl_gated_ffn(x, wg, wu, wd, out, saved=saved)
    ccl.ccl_gated_ffn_grad(dy, x, wg, wu, wd, saved, dx)
    xs, ys = x[ends].contiguous(), dy[ends].contiguous()
    o, d, s = torch.empty_like(xs), torch.empty_like(xs), torch.empty(2, 512, F, device=DEV)
    ccl.ccl_gated_ffn(xs, wg, wu, wd, o, saved=s)
    ccl.ccl_gated_ffn_grad(ys, xs, wg, wu, wd, s, d)
    assert torch.equal(saved[:, ends], s)
    # y and dx may be cut along K for few tokens: sums in another order, then one rounding to bf16
    for a, b in ((out[ends], o), (dx[ends], d)):
        assert float((a.double() - b.double()).norm()) <= 2.0 ** -9 * float(b.double().norm())
        assert bool(((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + 1e-4).all())
