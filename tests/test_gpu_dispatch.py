"""ccl_expert_order, ccl_dispatch, ccl_combine and ccl_combine_grad.  The order
and the copies are exact.  An fp32 sum of n products is good to n 2^-23 of the sum
of magnitudes, and an output is rounded once to its type."""
import numpy as np
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


def order_reference(ids, first, experts):
    flat = ids.cpu().numpy().astype(np.int64).reshape(-1) - first
    ok = (flat >= 0) & (flat < experts)
    at = np.nonzero(ok)[0]
    place = np.full(flat.size, -1, np.int64)
    place[at[np.argsort(flat[at], kind="stable")]] = np.arange(at.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=experts))]) if experts else np.zeros(1)
    return torch.from_numpy(offsets).to(DEV).to(I32), torch.from_numpy(place).to(DEV).to(I32).view(ids.shape)


def order(ids, experts, first=0, **kw):
    offsets = torch.full((experts + 1,), 55, device=DEV, dtype=I32)
    place = torch.full(ids.shape, 55, device=DEV, dtype=I32)
    ccl.ccl_expert_order(ids, offsets, place, first_expert=first, **kw)
    return offsets, place


# one choice; one CTA with few and all of its warps; experts that limit the warps; either side of 4096 and of 16384, where a cluster
# and several launches take over, the cluster with fewer threads than experts; several runs a CTA
@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 8), (7, 3, 5), (33, 1, 1024), (512, 8, 64), (500, 8, 700), (4096, 1, 1024), (4097, 1, 3), (1025, 4, 64),
                                   (2048, 8, 64), (16385, 1, 64), (5000, 3, 1024), (2001, 7, 400), (9001, 7, 400), (9000, 8, 1024), (100000, 2, 16),
                                   (1 << 20, 1, 1), (70001, 6, 333)])
def test_order(T, K, E):
    g = torch.Generator(device=DEV).manual_seed(T + E)
    ids = (torch.randn(T, K, generator=g, device=DEV).abs() * E / 3).to(I32).clamp_(max=E)  # uneven, E itself is none
    ids[torch.rand(T, K, generator=g, device=DEV) < 0.05] = -1
    for got, want in zip(order(ids, E), order_reference(ids, 0, E)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [100, 9000])
def test_order_of_a_ranks_experts(T):
    ids = torch.randint(-2, 70, (T, 3), device=DEV, dtype=I32)
    ids[0, 0], ids[1, 1] = -2 ** 31, 2 ** 31 - 1
    for first, n in ((0, 64), (16, 16), (63, 1), (-1, 3), (2 ** 31 - 1, 5), (-2 ** 31, 4)):
        for got, want in zip(order(ids, n, first), order_reference(ids, first, n)):
            assert torch.equal(got, want)


def test_order_of_nothing():
    for got, want in zip(order(torch.empty(0, 2, device=DEV, dtype=I32), 5), order_reference(torch.empty(0, 2), 0, 5)):
        assert torch.equal(got, want)
    offsets, place = order(torch.zeros(4, 2, device=DEV, dtype=I32), 0)
    assert offsets.tolist() == [0] and bool((place == -1).all())
    for T in (10, 9000):  # no choice has an expert; all have the same one
        ids = torch.full((T, 2), -1, device=DEV, dtype=I32)
        assert int(order(ids, 7)[0].abs().sum()) == 0 and bool((order(ids, 7)[1] == -1).all())
        ids.fill_(6)
        assert torch.equal(order(ids, 7)[1].flatten(), torch.arange(2 * T, device=DEV, dtype=I32))


def rows_like(n, dim, dtype, seed, lead=0, stride=None, fill=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    stride = stride or dim
    v = torch.zeros(lead + n * stride, device=DEV, dtype=dtype)[lead:].view(n, stride)[:, :dim]
    v.copy_(torch.randn(n, dim, generator=g, device=DEV) if fill is None else torch.full((n, dim), fill, device=DEV))
    return v


def places(T, K, seed, spare=3):
    """Distinct rows of T * K + spare for most choices, none for some."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    place = torch.randperm(T * K + spare, generator=g, device=DEV)[:T * K].view(T, K).to(I32)
    place[torch.rand(T, K, generator=g, device=DEV) < 0.2] = -1
    if T > 3:
        place[2] = -1                   # a token without any row
        place[3, 0] = T * K + spare     # just past the rows
        place[3, K - 1] = 2 ** 31 - 1
    return place, T * K + spare


# vectors of 32, 16 bytes and elements; several tokens a CTA; long rows; more choices than are loaded at a time
SHAPES = [(1, 1, 1), (1, 8, 4096), (5, 2, 64), (33, 3, 40), (100, 1, 8), (40, 5, 1031), (9, 4, 7168), (13, 32, 136), (300, 6, 12), (2, 2, 20000)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,K,D", SHAPES)
def test_dispatch(T, K, D, dtype):
    x = rows_like(T, D, dtype, 1)
    place, n = places(T, K, 2)
    rows = rows_like(n, D, dtype, 0, fill=9.0)
    want = rows.clone()
    ok = (place >= 0) & (place < n)
    want[place[ok].long()] = x[:, None].expand(T, K, D)[ok]
    ccl.ccl_dispatch(x, place, rows)
    assert torch.equal(rows, want)


def combine_reference(rows, place, weights):
    ok = (place >= 0) & (place < rows.shape[0])
    mine = rows.to(F64)[torch.where(ok, place, 0).long()]
    w = torch.where(ok, torch.ones_like(place, dtype=F64) if weights is None else weights.to(F64), 0.0)
    value = (mine * w[..., None]).sum(dim=1)
    return value, (place.shape[1] * 2.0 ** -23) * (mine.abs() * w.abs()[..., None]).sum(dim=1) + torch.finfo(rows.dtype).eps / 2 * value.abs() + 1e-37


def near(got, value, bound):
    bad = ~((got.to(F64) - value).abs() <= bound)
    assert not bool(bad.any()), (int(bad.sum()), float((got.to(F64) - value).abs().max()))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,K,D", SHAPES)
def test_combine_and_its_gradients(T, K, D, dtype):
    place, n = places(T, K, 3)
    rows, dy = rows_like(n, D, dtype, 4), rows_like(T, D, dtype, 5)
    w = torch.randn(T, K, device=DEV)
    ok = (place >= 0) & (place < n)
    w[~ok] = float("nan")  # the weight of a slot without a row does not count
    for weights in (w, None):
        out = rows_like(T, D, dtype, 0, fill=9.0)
        ccl.ccl_combine(rows, place, out, weights=weights)
        near(out, *combine_reference(rows, place, weights))
        grad_rows, grad_w = rows_like(n, D, dtype, 0, fill=9.0), torch.full((T, K), 9.0, device=DEV)
        want = grad_rows.to(F64)
        scaled = (torch.ones_like(w) if weights is None else w)[..., None].to(F64) * dy[:, None].to(F64)
        want[place[ok].long()] = scaled[ok]
        bound = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -24 * want.abs() + 1e-37
        ccl.ccl_combine_grad(dy, place, rows=rows, weights=weights, grad_rows=grad_rows, grad_weights=grad_w)
        near(grad_rows, want, bound)
        mine = rows.to(F64)[torch.where(ok, place, 0).long()] * dy[:, None].to(F64)
        near(grad_w, torch.where(ok, mine.sum(dim=2), 0.0), torch.where(ok, D * 2.0 ** -23 * mine.abs().sum(dim=2), 0.0) + 1e-37)
        alone = rows_like(n, D, dtype, 0, fill=9.0)
        ccl.ccl_combine_grad(dy, place, weights=weights, grad_rows=alone)
        assert torch.equal(alone, grad_rows)
        only = torch.full((T, K), 9.0, device=DEV)
        ccl.ccl_combine_grad(dy, place, rows=rows, weights=weights, grad_weights=only)
        assert torch.equal(only, grad_w)
        inplace = rows.clone()
        again = torch.full((T, K), 9.0, device=DEV)
        ccl.ccl_combine_grad(dy, place, rows=inplace, weights=weights, grad_rows=inplace, grad_weights=again)
        assert torch.equal(again, grad_w) and torch.equal(inplace[place[ok].long()], grad_rows[place[ok].long()])
        left = torch.ones(n, dtype=torch.bool, device=DEV)
        left[place[ok].long()] = False
        assert torch.equal(inplace[left], rows[left])


def test_combine_without_weights_is_dispatchs_gradient():
    """<dispatch(x), r> = <x, combine(r)> for every x and r: whole numbers, exact."""
    T, K, D = 50, 4, 24
    place, n = places(T, K, 6)
    x = torch.randint(-3, 4, (T, D), device=DEV).float()
    r = torch.randint(-3, 4, (n, D), device=DEV).float()
    rows, out = torch.zeros(n, D, device=DEV), torch.empty(T, D, device=DEV)
    ccl.ccl_dispatch(x, place, rows)
    ccl.ccl_combine(r, place, out)
    assert float((rows * r).sum()) == float((x * out).sum())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lead,stride", [(1, 96), (0, 97), (8, 104), (0, 100), (4, 96)])
def test_strides_and_alignment(dtype, lead, stride):
    T, K, D = 21, 3, 96
    place, n = places(T, K, 7)
    x = rows_like(T, D, dtype, 8, lead, stride)
    rows, plain = rows_like(n, D, dtype, 0, lead, stride, fill=2.0), rows_like(n, D, dtype, 0, fill=2.0)
    ccl.ccl_dispatch(x, place, rows)
    ccl.ccl_dispatch(x.contiguous(), place, plain)
    assert torch.equal(rows, plain)
    w = torch.rand(T, K, device=DEV)
    a, b = rows_like(T, D, dtype, 0, lead, stride), rows_like(T, D, dtype, 0)
    ccl.ccl_combine(rows, place, a, weights=w)
    ccl.ccl_combine(plain, place, b, weights=w)
    assert torch.equal(a, b)
    ga, gb = rows_like(n, D, dtype, 0, lead, stride), rows_like(n, D, dtype, 0)
    wa, wb = torch.empty(T, K, device=DEV), torch.empty(T, K, device=DEV)
    ccl.ccl_combine_grad(x, place, rows=rows, weights=w, grad_rows=ga, grad_weights=wa)
    ccl.ccl_combine_grad(x.contiguous(), place, rows=plain, weights=w, grad_rows=gb, grad_weights=wb)
    assert torch.equal(ga, gb)
    near(wa, wb.to(F64), 96 * 2.0 ** -22 * wb.abs().to(F64) + 1e-3)


def test_empty():
    e = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    i = lambda *s: torch.zeros(*s, device=DEV, dtype=I32)  # noqa: E731
    ccl.ccl_dispatch(e(0, 8), i(0, 2), e(5, 8))
    ccl.ccl_dispatch(e(3, 8), i(3, 2), e(0, 8))
    out = torch.full((3, 8), 5.0, device=DEV)
    ccl.ccl_combine(e(0, 8), i(3, 2), out)
    assert bool((out == 0).all())
    gw = torch.full((3, 2), 5.0, device=DEV)
    ccl.ccl_combine_grad(out, i(3, 2), rows=e(0, 8), grad_weights=gw, grad_rows=e(0, 8))
    assert bool((gw == 0).all())


def test_in_a_graph_and_on_another_stream():
    T, K, E, D = 3000, 2, 32, 64
    ids = torch.randint(-1, E, (T, K), device=DEV, dtype=I32)
    x, w = rows_like(T, D, BF16, 9), torch.rand(T, K, device=DEV)
    work = torch.empty(ccl.ccl_plan_expert_order_work_bytes(T, K, E), dtype=torch.uint8, device=DEV)

    def buffers():
        return [torch.zeros(E + 1, device=DEV, dtype=I32), torch.zeros(T, K, device=DEV, dtype=I32), torch.zeros(T * K, D, device=DEV, dtype=BF16),
                torch.zeros(T, D, device=DEV, dtype=BF16), torch.zeros(T * K, D, device=DEV, dtype=BF16), torch.zeros(T, K, device=DEV)]

    def go(b, **kw):
        offsets, place, rows, out, grad_rows, grad_w = b
        ccl.ccl_expert_order(ids, offsets, place, **kw)
        kw.pop("work", None)
        ccl.ccl_dispatch(x, place, rows, **kw)
        ccl.ccl_combine(rows, place, out, weights=w, **kw)
        ccl.ccl_combine_grad(x, place, rows=rows, weights=w, grad_rows=grad_rows, grad_weights=grad_w, **kw)
    want, other, captured = buffers(), buffers(), buffers()
    go(want, work=work)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    go(other, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(captured, work=work)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, captured):
        assert torch.equal(a, b) and torch.equal(a, c)
