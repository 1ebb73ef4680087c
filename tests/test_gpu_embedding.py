"""ccl_embedding and ccl_embedding_grad against plain 64-bit statements.

Lookup: one fp32 product and one round to the type, so bit for bit.
Gradient: a row's n tokens are added in fp32 (n - 1 additions, one product, one
more addition when accumulating) and rounded once, hence the bound
(n + 1) * 2^-24 * (scale * sum |dY| + |old|) + half a unit of the type."""
import math

import numpy as np
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def _ids(rng, n, rows, kind):
    if kind == "one":
        v = np.full(n, rows // 2)
    elif kind == "outside":
        v = np.where(rng.random(n) < 0.5, -1, rows + rng.integers(0, 5, n))
    elif kind == "zipf":
        v = np.minimum(rng.zipf(1.3, n) - 1, rows + 2)
    elif kind == "far":  # offsets that a 32-bit difference would wrap
        v = rng.choice(np.array([0, rows - 1, -2 ** 63, 2 ** 63 - 1, 2 ** 32, -2 ** 32]), n)
    else:
        v = rng.integers(-1, rows + 1, n)
    return torch.from_numpy(np.asarray(v, dtype=np.int64))


def _matrix(rng, n, d, dtype, stride=None, lead=0):
    """n x d normal values in rows `stride` apart, `lead` elements into the
    allocation; returns (view on the device, the same values in 64 bits)."""
    stride = stride or d
    big = torch.full((lead + n * stride + 8,), 7.0, dtype=dtype, device=DEV)
    view = big[lead:lead + n * stride].view(n, stride)[:, :d]
    host = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).to(dtype)
    view.copy_(host)
    return view, host.double(), big


SHAPES = [(1, 1, 1), (1, 5, 8), (3, 7, 129), (64, 300, 64), (65, 300, 40), (1000, 37, 1031), (2049, 5000, 256), (20000, 900, 72),
          (40, 257, 4096)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,rows,d", SHAPES)
def test_lookup(n, rows, d, dtype):
    rng = np.random.default_rng(n * 7 + d)
    table, _, _ = _matrix(rng, rows, d, dtype)
    ids = _ids(rng, n, rows, "uniform").to(DEV)
    out = torch.full((n, d), 9.0, dtype=dtype, device=DEV)
    scale = float(np.float32(math.sqrt(d) * 1.1))
    ccl.ccl_embedding(table, ids, out, scale=scale)
    ok = (ids >= 0) & (ids < rows)
    want = (table[torch.where(ok, ids, 0)].float() * torch.tensor(scale, device=DEV)).to(dtype)
    want[~ok] = 0
    assert torch.equal(out.view(torch.int16 if d and dtype == torch.bfloat16 else torch.int32),
                       want.view(torch.int16 if dtype == torch.bfloat16 else torch.int32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,stride,lead", [(64, 72, 0), (64, 64, 1), (61, 64, 3), (128, 256, 8)])
def test_lookup_strides_and_alignment(d, stride, lead, dtype):
    rng = np.random.default_rng(d + stride)
    table, _, _ = _matrix(rng, 50, d, dtype, stride, lead)
    out, _, whole = _matrix(rng, 33, d, dtype, stride + 8, lead)
    ids = _ids(rng, 33, 60, "uniform").to(DEV)
    guard = whole.clone()
    ccl.ccl_embedding(table, ids, out, scale=2.0, first_row=4)
    at = ids - 4
    ok = (at >= 0) & (at < 50)
    want = (table[torch.where(ok, at, 0)].float() * 2).to(dtype)
    want[~ok] = 0
    assert torch.equal(out, want)
    out.fill_(7.0)  # what lies between the rows was not touched
    guard[lead:lead + 33 * (stride + 8)].view(33, stride + 8)[:, :d] = 7.0
    assert torch.equal(whole, guard)


def test_shards_of_the_vocabulary_complete_each_other_by_allreduce():
    rng = np.random.default_rng(5)
    rows, d, n, ranks = 100, 24, 77, 4
    table, _, _ = _matrix(rng, rows, d, torch.float32)
    ids = _ids(rng, n, rows, "uniform").to(DEV)
    outs = [torch.empty(n, d, device=DEV) for _ in range(ranks)]
    for r in range(ranks):
        ccl.ccl_embedding(table[r * 25:(r + 1) * 25], ids, outs[r], first_row=r * 25)
    ccl.ccl_allreduce([o.view(-1) for o in outs])
    whole = torch.empty(n, d, device=DEV)
    ccl.ccl_embedding(table, ids, whole)
    for o in outs:
        assert torch.equal(o, whole)


def _check_grad(dy64, ids, first, rows, scale, got, old64, dtype):
    d = dy64.shape[1]
    want, mag = torch.zeros(rows, d, dtype=torch.float64), torch.zeros(rows, d, dtype=torch.float64)
    at = ids.cpu().numpy().astype(object) - first
    ok = np.array([0 <= int(v) < rows for v in at], dtype=bool)
    idx = torch.from_numpy(np.array([int(v) for v in at[ok]], dtype=np.int64))
    cnt = torch.zeros(rows, dtype=torch.float64).index_add_(0, idx, torch.ones(idx.numel(), dtype=torch.float64))
    want.index_add_(0, idx, dy64[torch.from_numpy(ok)] * scale)
    mag.index_add_(0, idx, (dy64[torch.from_numpy(ok)] * scale).abs())
    if old64 is not None:
        want += old64
        mag += old64.abs()
    bound = (cnt[:, None] + 1) * 2.0 ** -24 * mag + UNIT[dtype] * want.abs() * 1.01
    bad = (got.double().cpu() - want).abs() > bound
    assert not bool(bad.any()), "%d elements off" % int(bad.sum())
    return cnt


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["uniform", "zipf", "one", "outside", "far"])
@pytest.mark.parametrize("n,rows,d", SHAPES)
def test_gradient(n, rows, d, kind, dtype):
    rng = np.random.default_rng(n + 31 * d + rows)
    dy, dy64, _ = _matrix(rng, n, d, dtype)
    ids = _ids(rng, n, rows, kind).to(DEV)
    grad = torch.full((rows, d), 3.0, dtype=dtype, device=DEV)
    ccl.ccl_embedding_grad(dy, ids, grad, scale=1.5)
    cnt = _check_grad(dy64, ids, 0, rows, 1.5, grad, None, dtype)
    assert bool((grad.cpu()[cnt == 0] == 0).all())
    again = torch.full((rows, d), 4.0, dtype=dtype, device=DEV)
    ccl.ccl_embedding_grad(dy, ids, again, scale=1.5)
    assert torch.equal(grad, again)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,stride,lead,first", [(64, 72, 0, 0), (64, 64, 1, -3), (61, 64, 3, 10), (8, 8, 8, 2)])
def test_gradient_accumulates_in_place_and_keeps_what_is_between(d, stride, lead, first, dtype):
    rng = np.random.default_rng(d + lead)
    n, rows = 333, 60
    dy, dy64, _ = _matrix(rng, n, d, dtype, stride + 8, lead)
    grad, old64, whole = _matrix(rng, rows, d, dtype, stride, lead)
    before = whole.clone()
    ids = _ids(rng, n, rows + 5, "uniform").to(DEV)
    ids[ids % 7 == 0] = 1 << 40
    ccl.ccl_embedding_grad(dy, ids, grad, scale=0.5, first_row=first, accumulate=True)
    cnt = _check_grad(dy64, ids, first, rows, 0.5, grad, old64, dtype)
    assert torch.equal(grad.cpu()[cnt == 0], old64.to(dtype)[cnt == 0])
    before[lead:lead + rows * stride].view(rows, stride)[:, :d] = grad
    assert torch.equal(whole, before)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("kind", ["uniform", "one"])
@pytest.mark.parametrize("n", [127, 128, 129, 4095, 4096, 4097])
def test_gradient_where_ranking_by_counting_ends(n, kind, accumulate):
    rng = np.random.default_rng(n)
    rows, d = 700, 12
    dy, dy64, _ = _matrix(rng, n, d, torch.float32)
    grad, old64, _ = _matrix(rng, rows, d, torch.float32)
    ids = _ids(rng, n, rows, kind).to(DEV)
    ccl.ccl_embedding_grad(dy, ids, grad, scale=0.75, accumulate=accumulate)
    _check_grad(dy64, ids, 0, rows, 0.75, grad, old64 if accumulate else None, torch.float32)


@pytest.mark.parametrize("n", [500, 5000])
def test_gradient_of_more_rows_than_are_marked_at_a_time(n):
    # 16384 rows a CTA and two CTAs an SM at a time; here each marks a second range
    rows = 2 * torch.cuda.get_device_properties(0).multi_processor_count * 16500 + 7
    rng = np.random.default_rng(n)
    dy, dy64, _ = _matrix(rng, n, 2, torch.float32)
    ids = _ids(rng, n, rows, "uniform").to(DEV)
    grad = torch.full((rows, 2), 3.0, device=DEV)
    ccl.ccl_embedding_grad(dy, ids, grad)
    cnt = _check_grad(dy64, ids, 0, rows, 1.0, grad, None, torch.float32)
    assert bool((grad.cpu()[cnt == 0] == 0).all())


def test_no_tokens_and_no_rows():
    grad = torch.full((5, 8), 2.0, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    ccl.ccl_embedding_grad(torch.empty(0, 8, device=DEV), none, grad, accumulate=True)
    assert bool((grad == 2).all())
    ccl.ccl_embedding_grad(torch.empty(0, 8, device=DEV), none, grad)
    assert bool((grad == 0).all())
    ccl.ccl_embedding(grad, none, torch.empty(0, 8, device=DEV))
    out = torch.full((3, 8), 2.0, device=DEV)
    ccl.ccl_embedding(torch.empty(0, 8, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV), out)
    assert bool((out == 0).all())


def test_infinities_and_nan_stay_in_their_rows():
    dy = torch.ones(4, 8, device=DEV)
    dy[1] = float("inf")
    dy[2] = float("nan")
    ids = torch.tensor([0, 1, -1, 2], device=DEV)  # the NaN row is a padding token's
    grad = torch.empty(4, 8, device=DEV)
    ccl.ccl_embedding_grad(dy, ids, grad)
    assert grad[:, 0].tolist() == [1.0, float("inf"), 1.0, 0.0]
    out = torch.empty(4, 8, device=DEV)
    grad[3] = float("nan")
    ccl.ccl_embedding(grad, torch.tensor([-1, 0, 1, 3], device=DEV), out)
    assert bool((out[0] == 0).all()) and bool(torch.isnan(out[3]).all()) and bool(torch.isinf(out[2]).all())


def test_gradient_is_the_lookups_adjoint():
    """<lookup(E + D) - lookup(E), dY> = <dE, D>: the difference quotient of a
    linear map.  Integers keep every sum exact in fp32."""
    g = torch.Generator(device=DEV).manual_seed(3)
    E, D = (torch.randint(-4, 5, (50, 12), device=DEV, generator=g).float() for _ in range(2))
    dy = torch.randint(-4, 5, (200, 12), device=DEV, generator=g).float()
    ids = torch.randint(-2, 52, (200,), device=DEV, generator=g)
    a, b, grad = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(E)
    ccl.ccl_embedding(E + D, ids, a, scale=2.0)
    ccl.ccl_embedding(E, ids, b, scale=2.0)
    ccl.ccl_embedding_grad(dy, ids, grad, scale=2.0)
    assert float(((a - b) * dy).double().sum()) == float((grad * D).double().sum())


def test_another_stream_and_graph_replay():
    rng = np.random.default_rng(1)
    dy, dy64, _ = _matrix(rng, 300, 32, torch.float32)
    ids = _ids(rng, 300, 80, "zipf").to(DEV)
    grad = torch.empty(80, 32, device=DEV)
    work = torch.empty(ccl.ccl_plan_embedding_grad_work_bytes(300, 80, 32), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ccl.ccl_embedding_grad(dy, ids, grad, stream=s)  # its work buffer is allocated on s
    s.synchronize()
    _check_grad(dy64, ids, 0, 80, 1.0, grad, None, torch.float32)
    want = grad.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ccl.ccl_embedding_grad(dy, ids, grad, work=work)
    grad.fill_(5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(grad, want)
