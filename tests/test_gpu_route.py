"""ccl_route and ccl_route_grad against the formulas in 64 bits.

Bounds, with e = 2^-23: expf is good to 2 e, z - m to e |z - m| (a relative error
of exp of the same size), a sum of n positive terms to n e of itself.  So a
probability is good to c = (experts + 8 + 2 max|z - m|) e of itself, and lse to c
plus its own rounding."""
import math

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E32 = 2.0 ** -23


def make(T, E, K, dtype, seed=0, stride=None, lead=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 31 * T + E)
    stride = stride or E
    big = torch.zeros(lead + T * stride, device=DEV, dtype=dtype)
    z = big[lead:].view(T, stride)[:, :E]
    z.copy_(torch.randn(T, E, generator=g, device=DEV) * 2)
    return z, torch.randn(T, K, generator=g, device=DEV)


def route(z, K, normalize=True, valid=None, **kw):
    T, E = z.shape
    o = {"ids": torch.full((T, K), 77, device=DEV, dtype=I32), "weights": torch.full((T, K), 7.0, device=DEV), "lse": torch.full((T,), 7.0, device=DEV),
         "counts": torch.full((E + 1,), 77, device=DEV, dtype=I32), "load": torch.full((E,), 7.0, device=DEV),
         "importance": torch.full((E,), 7.0, device=DEV), "losses": torch.full((2,), 7.0, device=DEV)}
    ccl.ccl_route(z, *o.values(), normalize=normalize, valid=valid, **kw)
    return o


def reference(z, K, normalize, valid=None):
    """Values and bounds in 64 bits, of rows without NaN."""
    T, E = z.shape
    z = z.to(F64)
    m = z.amax(dim=1, keepdim=True)
    live = m[:, 0] > -math.inf
    if valid is not None:
        live &= valid != 0
    zz = torch.where(live[:, None], z - torch.where(live[:, None], m, 0.0), -math.inf)
    e = torch.where(live[:, None], zz.exp(), 0.0)
    p = e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)
    far = torch.where(e > 0, -zz, 0.0).amax(dim=1, keepdim=True)
    c = (E + 8 + 2 * far) * E32
    key = z + 0.0  # -0 and 0 tie
    order = key.sort(dim=1, descending=True, stable=True)
    ids = order.indices[:, :K]
    ok = live[:, None] & (order.values[:, :K] > -math.inf)
    w = torch.where(ok, p.gather(1, ids), 0.0)
    kept = w.sum(dim=1, keepdim=True)
    kept = torch.where(kept > 0, kept, 1.0)
    if normalize:
        w = w / kept
    n = int(live.sum())
    counts = torch.zeros(E + 1, device=DEV, dtype=torch.int64).index_add_(0, torch.where(ok, ids, E).flatten(), torch.ones(T * K, device=DEV, dtype=torch.int64))
    counts[E] = n
    load = counts[:E].to(F64) / max(1, int(counts[:E].sum()))
    importance = p.sum(dim=0) / max(n, 1)
    lse = torch.where(live, torch.where(live, m[:, 0], 0.0) + torch.log(e.sum(dim=1).clamp(min=1e-300)), 0.0)
    cl = torch.where(live, c[:, 0] + E32 * (lse.abs() + torch.where(live, m[:, 0].abs(), 0.0)), 0.0)
    cm = float(c.max()) + T * E32
    zl = (lse * lse).sum() / max(n, 1)
    return {"ids": (torch.where(ok, ids, -1).to(I32), None), "weights": (w, w * (2 * c + 4 * E32)), "lse": (lse, cl), "counts": (counts.to(I32), None),
            "load": (load, load * 2 * E32), "importance": (importance, importance * cm),
            "losses": (torch.stack([E * (load * importance).sum(), zl]),
                       torch.stack([E * (load * importance).sum() * (cm + (E + 4) * E32), (2 * lse.abs() * cl).sum() / max(n, 1) + zl * (T + 4) * E32])),
            "p": p, "live": live, "ok": ok, "c": c, "kept": kept}


def check(got, want, names=None):
    for k in names or got:
        value, bound = want[k]
        if bound is None:
            assert torch.equal(got[k], value), k
        else:
            # a value past fp32's range (the square of an lse of -3e38) is infinite there
            bad = ~(((got[k].to(F64) - value).abs() <= bound + 1e-37) | (torch.isinf(value.to(FP32)) & (got[k] == value.to(FP32))))
            assert not bool(bad.any()), (k, int(bad.sum()), float((got[k].to(F64) - value).abs().max()))


# each number of lanes and values a lane; odd counts; one expert; one token; several CTAs and the join
SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 16, 4), (17, 64, 6), (65, 64, 8), (64, 60, 2), (9, 65, 3), (33, 256, 8), (40, 255, 8), (70, 257, 12),
          (20, 1024, 32), (50, 640, 9), (1000, 64, 8), (5000, 256, 8), (7001, 37, 3), (20000, 16, 2), (300, 512, 16)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_forward(T, E, K, dtype):
    z, _ = make(T, E, K, dtype)
    for normalize in (True, False):
        check(route(z, K, normalize), reference(z, K, normalize))


def test_ties_go_to_the_lower_expert():
    z = torch.zeros(50, 64, device=DEV)
    z[1::2] = torch.randint(0, 3, (25, 64), device=DEV).float()
    z[0::4, ::3] = -0.0
    check(route(z, 8), reference(z, 8, True))
    z = torch.full((40, 300), 2.0, device=DEV, dtype=BF16)
    got = route(z, 9)
    assert torch.equal(got["ids"], torch.arange(9, device=DEV, dtype=I32).expand(40, 9))


@pytest.mark.parametrize("E,K", [(12, 4), (64, 8), (256, 8)])
def test_padding_and_masked_experts(E, K):
    T = 300
    z, gw = make(T, E, K, FP32, 5)
    valid = torch.rand(T, device=DEV) > 0.3
    z[7] = -math.inf                      # no expert at all
    z[8, 3:] = -math.inf                  # fewer than top
    z[:, 2] = -math.inf                   # an expert that no row but 9 may choose
    z[9] = torch.finfo(FP32).min          # the type's lowest value is a logit like any other
    others = torch.arange(T, device=DEV) != 9
    valid[7:10] = True
    dead = torch.nonzero(~valid)[0, 0]
    z[dead] = math.nan                    # what padding holds does not matter
    zz = torch.where(valid[:, None], z, -math.inf)
    got = route(z, K, True, valid)
    want = reference(zz, K, True)
    check(got, want)
    assert int(got["counts"][2]) == 1 and int(got["ids"][9, 2]) == 2 and int(got["counts"][E]) == int(valid.sum()) - 1
    gw[got["ids"] < 0] = math.nan         # nor what the slots without an expert get
    grad = torch.full((T, E), 3.0, device=DEV)
    ccl.ccl_route_grad(z, got["ids"], got["lse"], got["counts"], got["load"], gw, grad, balance=0.5, z=0.25)
    assert bool(torch.isfinite(grad).all()) and bool((grad[~valid] == 0).all()) and bool((grad[7] == 0).all()) and bool((grad[others, 2] == 0).all())


def test_a_nan_or_infinity_stays_in_its_row():
    z, _ = make(40, 64, 4, FP32, 8)
    clean = route(z, 4)
    z[3, 5], z[11, 60] = math.nan, math.inf
    got = route(z, 4)
    rest = [i for i in range(40) if i not in (3, 11)]
    for k in ("ids", "weights", "lse"):
        assert torch.equal(got[k][rest], clean[k][rest])
    assert bool(torch.isnan(got["weights"][[3, 11]]).all()) and int(got["ids"][3, 0]) == 5 and int(got["ids"][11, 0]) == 60
    assert int(got["ids"].min()) >= 0 and int(got["ids"].max()) < 64


def grads(z, o, gw, normalize, balance, zc, out=None):
    out = torch.full(z.shape, 3.0, device=DEV, dtype=z.dtype) if out is None else out
    ccl.ccl_route_grad(z, o["ids"], o["lse"], o["counts"], o["load"], gw, out, normalize=normalize, balance=balance, z=zc)
    return out


def reference_grad(z, o, gw, normalize, balance, zc, r):
    """(value, bound) from the router's own load, through the formula."""
    T, E = z.shape
    p, ok = r["p"], r["ok"]
    n = max(1, int(r["live"].sum()))
    ids = torch.where(ok, o["ids"], 0).long()
    gw = torch.where(ok, gw.to(F64), 0.0)
    size = gw.abs()
    if normalize:
        pt = torch.where(ok, p.gather(1, ids), 0.0)
        mean = (gw * pt).sum(dim=1, keepdim=True) / r["kept"]
        size = (gw.abs() + (gw.abs() * pt).sum(dim=1, keepdim=True) / r["kept"]) / r["kept"]
        gw = torch.where(ok, (gw - mean) / r["kept"], 0.0)
    pull = (balance * E / n * o["load"].to(F64)).expand(T, E)
    G = pull.scatter_add(1, ids, gw)
    S = pull.abs().scatter_add(1, ids, torch.where(ok, size, 0.0))
    lse = r["lse"][0]
    value = p * (G - (G * p).sum(dim=1, keepdim=True) + (2 * zc / n * lse)[:, None])
    # the kernel's p = exp(z - lse) is off by the error of lse and of z - lse too
    c = 4 * r["c"] + 2 * (r["lse"][1] + E32 * lse.abs())[:, None] + 8 * E32
    bound = p * (S + (S * p).sum(dim=1, keepdim=True) + (2 * abs(zc) / n * lse.abs())[:, None]) * c
    return value, bound + torch.finfo(z.dtype).eps / 2 * value.abs()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,E,K", SHAPES)
def test_gradient(T, E, K, dtype):
    z, gw = make(T, E, K, dtype, 2)
    for normalize, balance, zc in ((True, 0.7, 0.3), (False, 0.0, 0.0), (False, 0.2, 0.0)):
        o = route(z, K, normalize)
        check({"grad": grads(z, o, gw, normalize, balance, zc)}, {"grad": reference_grad(z, o, gw, normalize, balance, zc, reference(z, K, normalize))})


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(normalize):
    """The formula differentiated numerically in 64 bits, the choices and the
    load held: central differences of step h, whose error is h^2 times a third
    derivative (below 10 here)."""
    T, E, K, h = 6, 12, 3, 2.0 ** -10
    z, gw = make(T, E, K, FP32, 3)
    o = route(z, K, normalize)
    got = grads(z, o, gw, normalize, 0.5, 0.25).to(F64)

    def total(x):
        lp = torch.log_softmax(x, dim=1)
        w = lp.exp().gather(1, o["ids"].long())
        if normalize:
            w = w / w.sum(dim=1, keepdim=True)
        return (w * gw.to(F64)).sum() + 0.5 * E * (o["load"].to(F64) * lp.exp().mean(dim=0)).sum() + 0.25 * torch.logsumexp(x, dim=1).square().mean()
    for t in range(T):
        for j in range(E):
            d = torch.zeros(T, E, device=DEV, dtype=F64)
            d[t, j] = h
            q = float(total(z.to(F64) + d) - total(z.to(F64) - d)) / (2 * h)
            assert abs(q - float(got[t, j])) <= 10 * h * h + 1e-5


@pytest.mark.parametrize("lead,stride", [(1, 64), (0, 67), (4, 72)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_strides_and_alignment(dtype, lead, stride):
    z, gw = make(30, 64, 4, dtype, 4, stride, lead)
    o = route(z, 4)
    check(o, reference(z, 4, True))
    # rows without vectors are summed in another order: the same bound, not the same bits
    want = reference_grad(z, o, gw, True, 0.5, 0.1, reference(z, 4, True))
    rows = z._base[lead:].view(30, stride)
    got = rows.new_full((lead + 30 * stride,), 3.0)[lead:].view(30, stride)
    grads(z, o, gw, True, 0.5, 0.1, out=got[:, :64])
    check({"grad": got[:, :64]}, {"grad": want})
    assert bool((got[:, 64:] == 3).all())
    behind = rows[:, 64:].clone()
    assert torch.equal(grads(z, o, gw, True, 0.5, 0.1, out=z), got[:, :64])  # in place
    assert torch.equal(rows[:, 64:], behind)


def test_no_tokens():
    o = route(torch.empty(0, 16, device=DEV), 2)
    assert int(o["counts"].abs().sum()) == 0 and float(o["load"].abs().sum() + o["importance"].abs().sum() + o["losses"].abs().sum()) == 0
    grads(torch.empty(0, 16, device=DEV), o, torch.empty(0, 2, device=DEV), True, 1.0, 1.0)


def test_load_averaged_over_ranks_enters_the_gradient():
    z, gw = make(64, 32, 4, FP32, 6)
    o = route(z, 4)
    other = dict(o, load=torch.rand(32, device=DEV))
    r = reference(z, 4, True)
    check({"grad": grads(z, other, gw, True, 0.5, 0.0)}, {"grad": reference_grad(z, other, gw, True, 0.5, 0.0, r)})


def test_same_bits_each_time_in_a_graph_and_on_another_stream():
    z, gw = make(6000, 64, 4, BF16, 9)
    work = torch.empty(ccl.ccl_plan_route_work_bytes(6000, 64), dtype=torch.uint8, device=DEV)
    want = route(z, 4, work=work)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = route(z, 4, stream=s)
    s.synchronize()
    o = {k: torch.zeros_like(v) for k, v in want.items()}
    grad, want_grad = torch.zeros_like(z), grads(z, want, gw, True, 0.1, 0.1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ccl.ccl_route(z, *o.values(), work=work)
        ccl.ccl_route_grad(z, o["ids"], o["lse"], o["counts"], o["load"], gw, grad, balance=0.1, z=0.1)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], again[k]) and torch.equal(want[k], o[k]), k
    assert torch.equal(grad, want_grad)
