"""Rows of the distillation loss that the other tests' inputs leave out."""
import math

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [300, 50257])
def test_a_row_without_a_teacher_is_zero_whatever_its_weight(V, dtype):
    """0 by definition: an infinite or NaN weight must not make a NaN of it."""
    gen = torch.Generator(device=DEV).manual_seed(V)
    T, K = 6, 5
    logits = torch.randn(T, V, generator=gen, device=DEV).to(dtype)
    ids = torch.randint(0, V, (T, K), generator=gen, device=DEV)
    teacher = torch.randn(T, K, generator=gen, device=DEV)
    weights = torch.tensor([math.inf, math.nan, -math.inf, math.nan, 2.0, 1.0], device=DEV)
    ids[0], ids[1] = -1, V
    teacher[2:4] = -math.inf
    none = torch.tensor([True, True, True, True, False, False], device=DEV)
    loss, stats = torch.full((T,), 9.0, device=DEV), torch.empty(T, 2, device=DEV)
    for kept in (None, stats):
        ccl.ccl_distill_loss(logits, ids, teacher, loss.fill_(9), stats=kept, weights=weights)
        assert bool((loss[none] == 0).all()) and bool((loss[~none] > 0).all())
    grad = torch.full_like(logits, 9.0)
    ccl.ccl_distill_grad(logits, ids, teacher, stats, grad, weights=weights)
    assert bool((grad[none] == 0).all()) and bool((grad[~none] != 0).any(dim=1).all())
    later = grad.clone()
    ccl.ccl_distill_loss(logits, ids, teacher, loss.fill_(9), grad=grad.fill_(9), weights=weights)
    assert bool((loss[none] == 0).all()) and bool((loss[~none] > 0).all())
    assert torch.equal(grad[none], later[none])


@pytest.mark.parametrize("dtype,V", [(torch.float32, 140003), (torch.bfloat16, 300001)])
def test_rows_longer_than_a_cluster_holds_in_place(dtype, V):
    """What is read a second time is read before it is overwritten: the same
    bits as apart, in one call and from the kept statistics."""
    gen = torch.Generator(device=DEV).manual_seed(V)
    T, K = 3, 40
    logits = torch.randn(T, V, generator=gen, device=DEV).to(dtype)
    ids = torch.randint(0, V, (T, K), generator=gen, device=DEV)
    teacher = torch.randn(T, K, generator=gen, device=DEV)
    loss, again, stats = torch.empty(T, device=DEV), torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV)
    apart, later = torch.full_like(logits, 9.0), torch.full_like(logits, 9.0)
    ccl.ccl_distill_loss(logits, ids, teacher, loss, stats=stats, grad=apart)
    ccl.ccl_distill_grad(logits, ids, teacher, stats, later)
    one, two = logits.clone(), logits.clone()
    ccl.ccl_distill_loss(one, ids, teacher, again, grad=one)
    ccl.ccl_distill_grad(two, ids, teacher, stats, two)
    assert torch.equal(loss, again) and torch.equal(one, apart) and torch.equal(two, later)
    # and they are the definition's: rows sum to 0, and the listed entries differ from q by p
    q, p = torch.softmax(logits.double(), dim=1), torch.softmax(teacher.double(), dim=1)
    want = q.scatter_add(1, ids, -p)
    unit = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    assert bool(((apart.double() - want).abs() <= 2.0 ** -16 * (q + 1e-30) + (2.0 ** -16 + unit * 1.01) * want.abs() + 1e-38).all())
