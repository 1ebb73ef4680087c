"""ccl_act8_pack and ccl_act8_unpack against the definition in 64 bits: codes,
scales and the values that come back are equal to the bit."""
import math

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32, F64 = torch.bfloat16, torch.float32, torch.float64


def pow2(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def reference(x):
    """(codes, scales, values): blocks of 32 along the row."""
    n, c = x.shape
    w = -(-c // 32) * 32
    wide = torch.zeros(n, w, device=x.device, dtype=F64)
    wide[:, :c] = x.to(F64)
    b = wide.view(n, w // 32, 32)
    bad = ~torch.isfinite(b).all(dim=2)
    b = torch.where(bad[..., None], 0.0, b)
    frac, e = torch.frexp(b.abs().amax(dim=2) / 127)
    e = (e - (frac == 0.5).int()).clamp(-126, 121)
    e = torch.where(b.abs().amax(dim=2) == 0, -126, e)
    q = torch.round(b * pow2(-e[..., None])).clamp(-127, 127)
    value = (q * pow2(e[..., None])).masked_fill(bad[..., None], math.nan).view(n, w)[:, :c]
    return q.view(n, w).to(torch.int8), torch.where(bad, 255, e + 127).to(torch.uint8), value


def pack(x):
    n, c = x.shape
    w = ccl.ccl_plan_act8_width(c)
    codes, scales = torch.full((n, w), 99, device=DEV, dtype=torch.int8), torch.full((n, w // 32), 99, device=DEV, dtype=torch.uint8)
    ccl.ccl_act8_pack(x, codes, scales)
    return codes, scales


def check(x):
    codes, scales = pack(x)
    want = reference(x)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    for dtype in (BF16, FP32):
        back = torch.full(x.shape, 9.0, device=DEV, dtype=dtype)
        ccl.ccl_act8_unpack(codes, scales, back)
        assert torch.equal(back.to(F64).nan_to_num(nan=1e300), want[2].nan_to_num(nan=1e300))  # a bf16 number to the bit


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,c", [(1, 1), (1, 32), (3, 31), (5, 33), (7, 40), (2, 1001), (64, 136), (33, 4096), (1000, 72), (9, 2733)])
def test_values(n, c, dtype):
    g = torch.Generator(device=DEV).manual_seed(n + c)
    x = torch.randn(n, c, generator=g, device=DEV) * torch.exp(4 * torch.randn(n, 1, generator=g, device=DEV))
    x[n // 2, : c // 2] = 0
    check(x.to(dtype))


def test_edges_of_the_steps():
    """Blocks whose largest value is at, just under and just over 127 2^e, ties of
    the rounding, the smallest and largest numbers, infinities and NaN."""
    tops = []
    for e in (-140, -126, -125, -120, -20, 0, 1, 50, 119, 120, 121):
        for f in (127.0, 127.0 * (1 - 2 ** -23), 127.0 * (1 + 2 ** -23), 126.0, 64.0, 128.0, 1.0):
            v = f * 2.0 ** e
            tops.append(v if v < 3.4e38 else 3.4028234663852886e38)
    x = torch.zeros(len(tops), 32, device=DEV)
    top = torch.tensor(tops, device=DEV, dtype=F64).to(FP32)
    x[:, 5] = top
    x[:, 6] = -top
    step = torch.arange(26, device=DEV).float() - 12.5  # halves of a step: ties
    x[:, 6 + 0:32] = torch.where(torch.arange(26, device=DEV) == 0, -top[:, None], step * (top[:, None] / 127))
    check(x)
    check(x.to(BF16))
    x[3, 9], x[5, 0], x[8, 31] = math.nan, math.inf, -math.inf
    check(x)
    check(x.to(BF16))
    tiny = torch.full((2, 64), 2.0 ** -149, device=DEV)
    tiny[1, :32] = 2.0 ** -126
    check(tiny)


def test_error_is_half_a_step():
    x = torch.randn(100, 256, device=DEV)
    codes, scales = pack(x)
    back = torch.empty_like(x)
    ccl.ccl_act8_unpack(codes, scales, back)
    step = pow2(scales.to(torch.int64) - 127).repeat_interleave(32, dim=1)
    assert bool(((back.to(F64) - x.to(F64)).abs() <= step / 2).all())
    assert bool((step <= 2 * x.to(F64).view(100, 8, 32).abs().amax(dim=2).repeat_interleave(32, dim=1) / 127).all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("lead,stride", [(1, 72), (0, 73), (8, 80)])
def test_strides_and_alignment(dtype, lead, stride):
    big = torch.zeros(lead + 20 * stride, device=DEV, dtype=dtype)
    x = big[lead:].view(20, stride)[:, :72]
    x.copy_(torch.randn(20, 72, device=DEV))
    behind = big[lead:].view(20, stride)[:, 72:].clone()
    codes, scales = pack(x)
    want = reference(x)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    ccl.ccl_act8_unpack(codes, scales, x)
    assert torch.equal(x.to(F64), want[2]) and torch.equal(big[lead:].view(20, stride)[:, 72:], behind)


def test_empty_and_graph():
    ccl.ccl_act8_pack(torch.empty(0, 40, device=DEV), torch.empty(0, 64, device=DEV, dtype=torch.int8), torch.empty(0, 2, device=DEV, dtype=torch.uint8))
    x = torch.randn(50, 96, device=DEV, dtype=BF16)
    codes, scales = pack(x)
    c2, s2, back = torch.zeros_like(codes), torch.zeros_like(scales), torch.zeros_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ccl.ccl_act8_pack(x, c2, s2, stream=s)
    s.synchronize()
    assert torch.equal(c2, codes) and torch.equal(s2, scales)
    c2.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ccl.ccl_act8_pack(x, c2, s2)
        ccl.ccl_act8_unpack(c2, s2, back)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c2, codes) and torch.equal(back.to(F64), reference(x)[2])
