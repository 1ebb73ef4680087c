"""The expert-parallel operators on matrices whose offsets pass 32 bits (5 to 10
GB each): the rows at both ends against small calls on those rows alone, which the
other tests hold to the formulas."""
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def test_dispatch_and_combine():
    n, d, T, K = 600000, 8200, 40, 3  # rows of 9.8 GB, more than 2^32 elements
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, w = torch.randn(T, d, generator=gen, device=DEV).to(BF16), torch.rand(T, K, generator=gen, device=DEV)
    place = (torch.arange(T * K, device=DEV) * 2 + (torch.arange(T * K, device=DEV) % 2) * (n - 2 * T * K)).to(I32).view(T, K)
    small = torch.arange(T * K, device=DEV, dtype=I32).view(T, K)
    rows, few = torch.zeros(n, d, dtype=BF16, device=DEV), torch.zeros(T * K, d, dtype=BF16, device=DEV)
    ccl.ccl_dispatch(x, place, rows)
    ccl.ccl_dispatch(x, small, few)
    at = place.flatten().long()
    assert torch.equal(rows[at], few)
    a, b = torch.empty_like(x), torch.empty_like(x)
    ccl.ccl_combine(rows, place, a, weights=w)
    ccl.ccl_combine(few, small, b, weights=w)
    assert torch.equal(a, b)
    ga, gb = torch.empty(T, K, device=DEV), torch.empty(T, K, device=DEV)
    ccl.ccl_combine_grad(x, place, rows=rows, weights=w, grad_rows=rows, grad_weights=ga)
    ccl.ccl_combine_grad(x, small, rows=few, weights=w, grad_rows=few, grad_weights=gb)
    assert torch.equal(ga, gb) and torch.equal(rows[at], few)
    rows[at] = 0
    assert not bool(rows.view(torch.int16).any())  # nothing else was written


@pytest.mark.parametrize("cols", [8224, 8201])
def test_act8(cols):
    n = 600000  # codes of more than 2^32 bytes
    gen = torch.Generator(device=DEV).manual_seed(2)
    x = torch.zeros(n, cols, dtype=BF16, device=DEV)
    ends = [0, 1, 299999, n - 2, n - 1]
    x[ends] = torch.randn(5, cols, generator=gen, device=DEV).to(BF16)
    w = ccl.ccl_plan_act8_width(cols)
    big = (torch.empty(n, w, dtype=torch.int8, device=DEV), torch.empty(n, w // 32, dtype=torch.uint8, device=DEV))
    few = (torch.empty(5, w, dtype=torch.int8, device=DEV), torch.empty(5, w // 32, dtype=torch.uint8, device=DEV))
    ccl.ccl_act8_pack(x, *big)
    ccl.ccl_act8_pack(x[ends].contiguous(), *few)
    assert torch.equal(big[0][ends], few[0]) and torch.equal(big[1][ends], few[1])
    x[ends] = 0
    small = torch.empty(5, cols, dtype=BF16, device=DEV)
    ccl.ccl_act8_unpack(*big, x)
    ccl.ccl_act8_unpack(*few, small)
    assert torch.equal(x[ends], small)
    x[ends] = 0
    assert not bool(x.view(torch.int16).any())


def test_expert_ffn():
    """Two experts, the first with nearly all rows: x, out and grad_out pass 32
    bits in bytes, g, u, h, dg and du (600000 x 8192) in elements."""
    n, d, f = 600000, 4096, 8192
    gen = torch.Generator(device=DEV).manual_seed(3)
    rand = lambda *s: (torch.randn(*s, generator=gen, device=DEV) * s[-1] ** -0.5).to(BF16)  # noqa: E731
    wg, wu, wd = rand(2, f, d), rand(2, f, d), rand(2, d, f)
    ends = torch.cat([torch.arange(40, device=DEV), torch.arange(n - 60, n, device=DEV)])
    x, dy = torch.zeros(n, d, dtype=BF16, device=DEV), torch.zeros(n, d, dtype=BF16, device=DEV)
    x[ends], dy[ends] = rand(100, d) * 30, rand(100, d)

    def run(x, dy, counts):
        rows = x.shape[0]
        offsets = torch.tensor([0, counts[0], sum(counts)], device=DEV, dtype=I32)
        saved = (torch.empty(2, rows, f, dtype=torch.int8, device=DEV), torch.empty(2, rows, f // 32, dtype=torch.uint8, device=DEV))
        out, dx = torch.empty_like(x), torch.empty_like(x)
        grads = [torch.empty_like(w) for w in (wg, wu, wd)]
        ccl.ccl_expert_ffn(x, offsets, wg, wu, wd, out, saved=saved)
        ccl.ccl_expert_ffn_grad(dy, x, offsets, wg, wu, wd, saved, dx, *grads)
        return out, dx, grads, saved
    out, dx, grads, saved = run(x, dy, (n - 20, 20))
    few = run(x[ends].contiguous(), dy[ends].contiguous(), (80, 20))
    # the few rows go through another kernel, whose sums of products are in another order: to the rounding of g, u (8 bits) and of the output
    for a, b in ((out[ends], few[0]), (dx[ends], few[1]), *zip(grads, few[2])):
        assert float((a.float() - b.float()).norm()) <= 2.0 ** -8 * float(b.float().norm())
    assert float((saved[0][:, ends].float() - few[3][0].float()).abs().max()) <= 1
    assert torch.equal(saved[1][:, ends], few[3][1])
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[ends] = False
    assert not bool(out[rest].any()) and not bool(dx[rest].any())
    assert ccl.ccl_gated_ffn_timeouts() == 0
