"""ccl_route_grad on logits far from zero, against the formula in 64 bits: a common
offset of a row's logits changes neither the probabilities nor what the balance loss
and the weights pull, so the bounds do not grow with it.

With e = 2^-23: expf is good to 2 + 1.2 d units at d = |z - m|, and the rounding of
z - m adds d / 2, so a term is good to (2 + 2 d) e of itself; their sum of E, the
quotient and the product add (E + 3) e.  A probability is then good to c = (E + 8 + 4
far) e of itself, far being the largest d of a term above 0.  A gradient is a product
of one, c, with sums of their products and quotients: the weights' gradients, when
normalised, have two more of them, the inner product one, and each sum its length in
e: 4 c covers both.  The z loss alone looks at lse itself, which is rounded to fp32."""
import math

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E32 = 2.0 ** -23


def route(z, K, normalize):
    T, E = z.shape
    o = [torch.empty(T, K, device=DEV, dtype=I32), torch.empty(T, K, device=DEV), torch.empty(T, device=DEV), torch.empty(E + 1, device=DEV, dtype=I32),
         torch.empty(E, device=DEV), torch.empty(E, device=DEV), torch.empty(2, device=DEV)]
    ccl.ccl_route(z, *o, normalize=normalize)
    return o


def check(z, K, gw, normalize, balance, zc, load=None):
    T, E = z.shape
    ids, weights, lse, counts, own_load, _, _ = route(z, K, normalize)
    load = own_load if load is None else load
    grad = torch.full((T, E), 3.0, device=DEV, dtype=z.dtype)
    ccl.ccl_route_grad(z, ids, lse, counts, load, gw, grad, normalize=normalize, balance=balance, z=zc)
    x = z.to(F64)
    m = x.amax(dim=1, keepdim=True)
    p = (x - m).exp()
    far = torch.where(p > 0, m - x, 0.0).amax(dim=1, keepdim=True)
    p = p / p.sum(dim=1, keepdim=True)
    c = (E + 8 + 4 * far) * E32
    at, g = ids.long(), gw.to(F64)
    kept = p.gather(1, at).sum(dim=1, keepdim=True)
    w = p.gather(1, at) / (kept if normalize else 1.0)
    assert bool(((weights.to(F64) - w).abs() <= 2 * c * w + 1e-37).all())
    size = g.abs()
    if normalize:
        size = (g.abs() + (g.abs() * w).sum(dim=1, keepdim=True)) / kept
        g = (g - (g * w).sum(dim=1, keepdim=True)) / kept
    pull = (balance * E / T * load.to(F64)).expand(T, E)
    G, S = pull.scatter_add(1, at, g), pull.abs().scatter_add(1, at, size)
    true_lse = m[:, 0] + torch.log((x - m).exp().sum(dim=1))
    zterm = 2 * zc / T * true_lse[:, None]
    value = p * (G - (G * p).sum(dim=1, keepdim=True) + zterm)
    bound = p * (S + (S * p).sum(dim=1, keepdim=True) + zterm.abs()) * 4 * c + p * (2 * zc / T) * (c + 2 * E32 * true_lse.abs()[:, None])
    bad = ~((grad.to(F64) - value).abs() <= bound + torch.finfo(z.dtype).eps / 2 * value.abs() + 1e-37)
    assert not bool(bad.any()), (int(bad.sum()), float((grad.to(F64) - value).abs().max()), float(value.abs().max()))
    return grad, value


def logits(T, E, dtype, offset, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + T + E)
    z = torch.randn(T, E, generator=g, device=DEV) * 2 + offset
    return z.to(dtype), g


# every number of lanes and values a lane
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("T,E,K", [(30, 8, 2), (30, 16, 4), (65, 64, 8), (9, 37, 3), (33, 256, 8), (20, 500, 12), (7, 1000, 32)])
def test_a_common_offset(T, E, K, dtype, normalize):
    for offset in (100.0, -1e3, 1e4, -1e4, 1e6, -1e9, 1e30):
        z, g = logits(T, E, dtype, offset)
        gw = torch.randn(T, K, generator=g, device=DEV) / T
        check(z, K, gw, normalize, 0.7, 0.0)
        check(z, K, torch.zeros_like(gw), normalize, 1e-2, 0.0, torch.rand(E, generator=g, device=DEV))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("E,K", [(8, 2), (64, 4), (256, 8), (512, 8), (1024, 8)])
def test_rows_of_one_finite_value_are_even(E, K, dtype):
    """A token masked with -1e9, the type's lowest or highest value instead of -inf:
    every expert has 1 / E, the balance loss pulls it by that much and no more."""
    for value in (-1e9, torch.finfo(dtype).min, torch.finfo(dtype).max, 1e9, 0.0):
        z, g = logits(12, E, dtype, 0.0, 3)
        z[5] = value
        load = torch.rand(E, generator=g, device=DEV)
        grad, want = check(z, K, torch.zeros(12, K, device=DEV), True, 1e-2, 0.0, load)
        assert float(grad[5].abs().max()) <= 1.01 * float(want[5].abs().max())
        check(z, K, torch.randn(12, K, generator=g, device=DEV), False, 0.0, 0.0)
        check(z, K, torch.randn(12, K, generator=g, device=DEV), True, 0.5, 0.0)


@pytest.mark.parametrize("E,K", [(64, 4), (256, 8)])
def test_the_z_loss_far_from_zero(E, K):
    for offset in (30.0, -300.0, 1e4):
        z, g = logits(40, E, FP32, offset, 4)
        check(z, K, torch.randn(40, K, generator=g, device=DEV), True, 0.1, 1e-3)


@pytest.mark.parametrize("E,K", [(64, 4), (300, 8)])
def test_weights_and_their_gradient_agree(E, K):
    """Not normalised, one weight's gradient by its own logit is w (1 - w): the w that
    the forward pass gave."""
    z, _ = logits(50, E, FP32, 5e3, 5)
    ids, w, lse, counts, load, _, _ = route(z, K, False)
    gw = torch.zeros(50, K, device=DEV)
    gw[:, 0] = 1
    grad = torch.empty_like(z)
    ccl.ccl_route_grad(z, ids, lse, counts, load, gw, grad, normalize=False)
    want = (w[:, 0] * (1 - w[:, 0])).to(F64)
    got = grad.gather(1, ids[:, :1].long())[:, 0].to(F64)
    assert bool(((got - want).abs() <= 8 * E32 * w[:, 0]).all())
    rest = grad.to(F64).sum(dim=1)  # p sums to 1, so a row's gradient sums to 0
    assert float((rest.abs() - (E + 40) * E32 * grad.to(F64).abs().sum(dim=1)).max()) <= 0


def test_infinities_and_nan_stay_in_their_rows():
    z, g = logits(20, 64, FP32, 1e4, 6)
    gw = torch.randn(20, 4, generator=g, device=DEV)
    load = torch.rand(64, generator=g, device=DEV)

    def grads(z):
        ids, _, lse, counts, _, _, _ = route(z, 4, True)
        out = torch.full_like(z, 3.0)
        ccl.ccl_route_grad(z, ids, lse, counts, load, gw, out, balance=0.5)
        return out
    clean = grads(z)
    z[3, 5], z[4], z[6, 7], z[8, :61] = math.nan, math.nan, math.inf, -math.inf
    got = grads(z)
    rest = [i for i in range(20) if i not in (3, 4, 6, 8)]
    assert torch.equal(got[rest], clean[rest])
    assert bool(torch.isnan(got[[3, 4, 6]]).all()) and bool((got[8, :61] == 0).all()) and bool(torch.isfinite(got[8]).all())
