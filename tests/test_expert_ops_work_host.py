"""A work buffer planned for a rank's largest batch serves every smaller one, as
batches vary from call to call: what the planners ask for, without a GPU."""
import random

import pytest

import ring_allreduce_rank_gb300 as ccl

@pytest.fixture(scope="module", autouse=True)
def _built():
    from ring_allreduce_rank_gb300 import build
    build.build()
    ccl.lib()


def _counts(most, around, seed):
    """1 to most: the smallest, both sides of `around` and its multiples, and others on a logarithmic scale."""
    rng = random.Random(seed)
    n = set(range(1, 200)) | {int(2 ** rng.uniform(0, most.bit_length())) for _ in range(3000)}
    for a in around:
        for k in range(1, 40):
            n |= {k * a - 1, k * a, k * a + 1}
    return sorted(k for k in n if 1 <= k <= most)


@pytest.mark.parametrize("experts", [1, 8, 63, 64, 65, 100, 256, 700, 1024])
def test_the_orders_work_never_falls_as_tokens_grow(experts):
    for top in (1, 3, 8):
        before = (0, 0)
        for n in _counts((1 << 31) // top - 1, (4096, 16384, 77824, 8 * 152 * 64, 8 * 152 * 96), experts):
            size = ccl.ccl_plan_expert_order_work_bytes(n, top, experts)
            assert size >= before[0], (n, before)
            before = size, n


@pytest.mark.parametrize("experts", [1, 64, 256, 257, 512, 1000])
def test_the_routers_work_never_falls_as_tokens_grow(experts):
    before = (0, 0)
    for n in _counts(1 << 24, (8, 32, 152, 304, 1216, 4864), experts):
        size = ccl.ccl_plan_route_work_bytes(n, experts)
        assert size >= before[0], (n, before)
        before = size, n
