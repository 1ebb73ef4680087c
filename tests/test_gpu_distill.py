"""ccl_distill_loss and ccl_distill_grad against the definition in 64 bits.

Bounds: the exponential is good to 2^-22 and its argument's product adds at
most |x| 2^-24 (|x| < 40 where a term matters), a row's sum adds under 100
roundings, so q and p are good to 2^-17 of themselves; the loss adds those of
its logarithms.  TOL = 2^-16 covers a quotient of two such values."""
import math

import numpy as np
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL = 2.0 ** -16
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def reference(logits, ids, teacher, weights, tau):
    """(loss, grad, magnitude of the loss's terms, q + p) in 64 bits."""
    s = logits.double().cpu() / tau
    T, V = s.shape
    ids, t = ids.cpu(), teacher.double().cpu() / tau
    w = torch.ones(T, dtype=torch.float64) if weights is None else weights.double().cpu()
    loss, grad = torch.zeros(T, dtype=torch.float64), torch.zeros(T, V, dtype=torch.float64)
    mag, qp = torch.zeros(T, dtype=torch.float64), torch.zeros(T, V, dtype=torch.float64)
    for r in range(T):
        ok = (ids[r] >= 0) & (ids[r] < V)
        tv, iv = t[r][ok], ids[r][ok]
        if w[r] == 0 or tv.numel() == 0 or bool((tv == -math.inf).all()):
            continue
        p = torch.softmax(tv, 0)
        z = s[r] - s[r].max()  # first, or a row of huge values loses its logarithm
        logq = z - torch.log(torch.exp(z).sum())
        q = logq.exp()
        on = ~(p == 0)
        terms = p[on] * (p[on].log() - logq[iv[on]])
        loss[r] = w[r] * terms.sum()
        mag[r] = w[r].abs() * (p[on] * (p[on].log().abs() + logq[iv[on]].abs() + 1)).sum()
        ps = torch.zeros(V, dtype=torch.float64).index_add_(0, iv, p)
        grad[r] = w[r] / tau * (q - ps)
        qp[r] = (w[r] / tau).abs() * (q + ps)
    return loss, grad, mag, qp


def inputs(T, V, K, dtype, seed, stride=None, lead=0):
    rng = np.random.default_rng(seed)
    stride = stride or V
    big = torch.full((lead + T * stride + 8,), 7.0, dtype=dtype, device=DEV)
    logits = big[lead:lead + T * stride].view(T, stride)[:, :V]
    logits.copy_(torch.from_numpy(rng.standard_normal((T, V)).astype(np.float32) * 2))
    ids = torch.from_numpy(rng.integers(0, V, (T, K))).to(DEV)
    teacher = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32) * 3).to(DEV)
    weights = torch.from_numpy(rng.random(T).astype(np.float32) + 0.5).to(DEV)
    return logits, ids, teacher, weights, big


def check(logits, ids, teacher, weights, tau, loss, grad=None, ref=None):
    want, dwant, mag, qp = ref or reference(logits, ids, teacher, weights, tau)
    assert bool(((loss.double().cpu() - want).abs() <= TOL * mag).all())
    if grad is not None:
        bound = TOL * qp + UNIT[grad.dtype] * 1.01 * (dwant.abs() + TOL * qp) + 1e-38
        bad = (grad.double().cpu() - dwant).abs() > bound
        assert not bool(bad.any()), "%d gradients off" % int(bad.sum())


def all_forms(logits, ids, teacher, weights, tau):
    T, V = logits.shape
    ref = reference(logits, ids, teacher, weights, tau)
    loss, stats = torch.full((T,), 9.0, device=DEV), torch.empty(T, 2, device=DEV)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, weights=weights, temperature=tau)
    check(logits, ids, teacher, weights, tau, loss, ref=ref)
    loss.fill_(9)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, stats=stats, weights=weights, temperature=tau)
    check(logits, ids, teacher, weights, tau, loss, ref=ref)
    grad = torch.full((T, V), 9.0, dtype=logits.dtype, device=DEV)
    ccl.ccl_distill_grad(logits, ids, teacher, stats, grad, weights=weights, temperature=tau)
    check(logits, ids, teacher, weights, tau, loss, grad, ref=ref)
    one, oneg = torch.full((T,), 9.0, device=DEV), torch.full((T, V), 9.0, dtype=logits.dtype, device=DEV)
    ccl.ccl_distill_loss(logits, ids, teacher, one, grad=oneg, weights=weights, temperature=tau)
    check(logits, ids, teacher, weights, tau, one, oneg, ref=ref)
    return loss, grad


SHAPES = [(1, 1, 1), (3, 5, 2), (2, 7, 9), (5, 1000, 17), (4, 1001, 64), (2, 50257, 20), (300, 333, 5), (1, 131072, 1024), (3, 70001, 300)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,K", SHAPES)
def test_loss_and_gradient(T, V, K, dtype):
    logits, ids, teacher, weights, _ = inputs(T, V, K, dtype, T + V + K)
    all_forms(logits, ids, teacher, weights, 1.7)
    all_forms(logits, ids, teacher, None, 1.0)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 140003), (torch.bfloat16, 300000)])
def test_rows_longer_than_the_registers_of_a_cluster(dtype, V):
    logits, ids, teacher, weights, _ = inputs(2, V, 50, dtype, 3)
    all_forms(logits, ids, teacher, weights, 2.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,stride,lead", [(1000, 1008, 0), (1000, 1000, 1), (997, 1003, 3), (64, 72, 5)])
def test_strides_alignment_and_in_place(V, stride, lead, dtype):
    T, K, tau = 6, 12, 1.3
    logits, ids, teacher, weights, whole = inputs(T, V, K, dtype, V + lead, stride, lead)
    ref = reference(logits, ids, teacher, weights, tau)
    loss, stats = torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV)
    apart = torch.empty(T, V, dtype=dtype, device=DEV)  # another alignment than the logits
    ccl.ccl_distill_loss(logits, ids, teacher, loss, stats=stats, grad=apart, weights=weights, temperature=tau)
    check(logits, ids, teacher, weights, tau, loss, apart, ref=ref)
    keep = whole.clone()
    ccl.ccl_distill_loss(logits, ids, teacher, loss, grad=logits, weights=weights, temperature=tau)
    check(None, None, None, None, tau, loss, logits, ref=ref)
    assert torch.equal(logits, apart)
    after, whole_after = logits.clone(), whole.clone()
    whole.copy_(keep)
    ccl.ccl_distill_grad(logits, ids, teacher, stats, logits, weights=weights, temperature=tau)
    check(None, None, None, None, tau, loss, logits, ref=ref)
    # what lies between the rows keeps its bits
    view = whole_after[lead:lead + T * stride].view(T, stride)
    assert torch.equal(view[:, V:], keep[lead:lead + T * stride].view(T, stride)[:, V:])
    assert torch.equal(whole_after[:lead], keep[:lead]) and torch.equal(view[:, :V], after)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_entries_rows_and_weights(dtype):
    logits, ids, teacher, weights, _ = inputs(8, 500, 6, dtype, 11)
    ids[0] = -1                       # no teacher
    teacher[1] = -math.inf            # a teacher of nothing
    ids[2, 3:] = torch.tensor([-1, 500, 2 ** 40], device=DEV)
    teacher[2, 3:] = math.nan         # what a masked entry holds does not matter
    weights[3] = 0
    logits[3, 10] = math.nan          # nor what a row of weight 0 holds
    logits[4, 100:] = -math.inf       # a masked part of the vocabulary
    ids[4] = torch.arange(6, device=DEV)
    ids[5] = 7                        # one id in every entry
    teacher[6, 1:] = -math.inf
    logits[7] = torch.finfo(dtype).min  # a row of the type's lowest value: uniform
    teacher[7] = torch.finfo(torch.float32).min
    clean = logits.clone()
    clean[3] = 0
    ref = reference(clean, ids, teacher, weights, 1.5)
    loss, grad = torch.empty(8, device=DEV), torch.full((8, 500), 9.0, dtype=dtype, device=DEV)
    stats = torch.empty(8, 2, device=DEV)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, grad=grad, weights=weights, temperature=1.5)
    check(None, None, None, None, 1.5, loss, grad, ref=ref)
    assert loss[[0, 1, 3]].tolist() == [0.0, 0.0, 0.0] and bool((grad[[0, 1, 3]] == 0).all())
    assert bool((grad[4, 100:] == 0).all())
    grad.fill_(9)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, stats=stats, weights=weights, temperature=1.5)
    ccl.ccl_distill_grad(logits, ids, teacher, stats, grad, weights=weights, temperature=1.5)
    check(None, None, None, None, 1.5, loss, grad, ref=ref)
    assert loss[3].item() == 0 and bool((grad[3] == 0).all())
    # a teacher id outside the student's vocabulary mask: infinite loss, finite gradient
    ids[4, 0] = 200
    ccl.ccl_distill_loss(logits, ids, teacher, loss, grad=grad, weights=weights, temperature=1.5)
    assert loss[4].item() == math.inf and bool(torch.isfinite(grad[4]).all())
    # a NaN teacher logit of a valid id reaches the loss of its row alone
    teacher[5, 2] = math.nan
    ccl.ccl_distill_loss(logits, ids, teacher, loss, weights=weights, temperature=1.5)
    assert torch.isnan(loss).tolist() == [False] * 5 + [True, False, False]


def test_stats_are_the_rows_maximum_and_sum():
    logits, ids, teacher, weights, _ = inputs(7, 5003, 4, torch.float32, 2)
    ids[2] = -1
    weights[3] = 0  # the stats are kept for rows without a loss too
    loss, stats = torch.empty(7, device=DEV), torch.empty(7, 2, device=DEV)
    grad = torch.empty_like(logits)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, stats=stats, grad=grad, weights=weights, temperature=2.5)
    x = logits.double()
    m = x.max(dim=1).values
    z = torch.exp((x - m[:, None]) / 2.5).sum(dim=1)
    assert torch.equal(stats[:, 0].double(), m)
    assert bool(((stats[:, 1].double() - z).abs() <= TOL * z).all())


def test_no_teacher_entries_and_no_rows():
    logits = torch.randn(3, 40, device=DEV)
    none = torch.empty(3, 0, dtype=torch.int64, device=DEV)
    loss, grad = torch.full((3,), 5.0, device=DEV), torch.full((3, 40), 5.0, device=DEV)
    ccl.ccl_distill_loss(logits, none, torch.empty(3, 0, device=DEV), loss, grad=grad)
    assert bool((loss == 0).all()) and bool((grad == 0).all())
    empty = torch.empty(0, 40, device=DEV)
    ccl.ccl_distill_loss(empty, torch.empty(0, 4, dtype=torch.int64, device=DEV), torch.empty(0, 4, device=DEV),
                         torch.empty(0, device=DEV), grad=torch.empty(0, 40, device=DEV))


def test_gradient_against_differences():
    """The loss's central difference along random directions; the quotient's
    own error is h^2 times the third derivative (below 1 here) plus the
    losses' rounding over h."""
    T, V, K, tau, h = 4, 300, 8, 1.5, 2.0 ** -6
    logits, ids, teacher, weights, _ = inputs(T, V, K, torch.float32, 8)
    loss, grad = torch.empty(T, device=DEV), torch.empty(T, V, device=DEV)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, grad=grad, weights=weights, temperature=tau)
    for k in range(4):
        d = torch.randn(T, V, device=DEV, generator=torch.Generator(device=DEV).manual_seed(k))
        up, down = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        ccl.ccl_distill_loss(logits + h * d, ids, teacher, up, weights=weights, temperature=tau)
        ccl.ccl_distill_loss(logits - h * d, ids, teacher, down, weights=weights, temperature=tau)
        quotient = (up - down).double() / (2 * h)
        along = (grad.double() * d).sum(dim=1)
        assert bool(((quotient - along).abs() <= 4 * h * h + 8 * TOL / h).all())


def test_same_bits_each_time_and_in_a_graph():
    logits, ids, teacher, weights, _ = inputs(40, 9001, 30, torch.bfloat16, 4)
    loss, grad = torch.empty(40, device=DEV), torch.empty_like(logits)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, grad=grad, weights=weights)
    a, b = loss.clone(), grad.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ccl.ccl_distill_loss(logits, ids, teacher, loss, grad=grad, weights=weights)
    loss.fill_(1)
    grad.fill_(1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, a) and torch.equal(grad, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ccl.ccl_distill_loss(logits, ids, teacher, loss, grad=grad, weights=weights, stream=s)
    s.synchronize()
    assert torch.equal(loss, a) and torch.equal(grad, b)
