"""A work buffer planned for a rank's largest batch serves every smaller one, as
batches vary from call to call.  Without a GPU: what the planners ask for, and the C
entries' check of the buffer, in a child process that sees no GPU, on fake pointers
that are never dereferenced."""
import os
import random
import subprocess
import sys

import pytest

import ring_allreduce_rank_gb300 as ccl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, CUDA = 1, 4
T40 = 1 << 40

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


def _ffn(L, n, e, d, f, nbytes):
    return L.ccl_expert_ffn(T40, 7 * T40, 2 * T40, 3 * T40, 4 * T40, n, e, d, f, 1, 0, 5 * T40, None, None, 6 * T40, nbytes, None)


def _ffn_grad(L, n, e, d, f, nbytes):
    return L.ccl_expert_ffn_grad(T40, 2 * T40, None, None, 3 * T40, 4 * T40, 5 * T40, 6 * T40, 7 * T40, 8 * T40, n, e, d, f, 1, 0, 0, 9 * T40, 10 * T40, 11 * T40,
                                 12 * T40, 13 * T40, nbytes, None)


def _order(L, n, top, e, nbytes):
    return L.ccl_expert_order(T40, n, top, 0, e, 2 * T40, 3 * T40, 4 * T40, nbytes, None)


def accepted(L):
    """Calls that pass their checks go on to a launch, which fails here."""
    plan = ccl.ccl_plan_expert_ffn_work_bytes
    for e, d, f in ((1, 4096, 4096), (8, 4096, 11008), (64, 2048, 1408), (5, 1001, 733), (3, 130, 77), (1, 64, 8192)):
        for most in (1, 2, 4, 16, 63 * e, 64 * e, 64 * e + 1, 64 * e + 5, 70 * e, 100 * e):
            forward, both = plan(most, e, d, f), plan(most, e, d, f, backward=True)
            for n in sorted({1, 2, 3, 5, 8, 13, 21, 34, 55, 89, e, 2 * e, 16 * e, 32 * e, 63 * e, 64 * e, 64 * e + 1, most - 1, most}):
                if 1 <= n <= most:
                    assert _ffn(L, n, e, d, f, forward) == CUDA, (n, most, e, d, f)
                    assert _ffn(L, n, e, d, f, both) == CUDA, (n, most, e, d, f)
                    assert _ffn_grad(L, n, e, d, f, both) == CUDA, (n, most, e, d, f)
    # what no call can do without is still asked for: h, and for odd widths the copies
    assert _ffn(L, 64, 1, 4096, 4096, 64 * 4096 * 2) == CUDA and _ffn(L, 64, 1, 4096, 4096, 64 * 4096 * 2 - 1) == INVALID
    assert _ffn(L, 4, 1, 12, 32, 4 * 32 * 2 + 4 * 16 * 2 + 2 * 32 * 16 * 2 - 1) == INVALID
    for e in (8, 64, 300):
        for most in (77824, 77825, 100000):
            nbytes = ccl.ccl_plan_expert_order_work_bytes(most, 1, e)
            for n in (16385, 20000, 60000, 77824, most):
                assert n > most or _order(L, n, 1, e, nbytes) == CUDA, (n, most, e)


def test_a_larger_batchs_buffer_is_accepted():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    res = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "accepted ok" in res.stdout


if __name__ == "__main__":
    accepted(ccl.lib())
    print("accepted ok")
