"""ccl_gated_ffn and ccl_gated_ffn_grad against the formulas in 64 bits.

Bounds, with r = 2^-8 (bf16's unit roundoff: 8 significant bits): an fp32 sum of n
products is good to n 2^-23 of the sum of magnitudes, an activation to 2^-18 of
itself; h, dg and du carry those errors of their factors and one rounding r,
which the next product sums; each output is rounded once more."""
import math

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
R = 2.0 ** -8
ACT = 2.0 ** -18


def act64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


def reference(x, wg, wu, wd, dy, act):
    """{name: (value, bound)} in 64 bits."""
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    (T, D), F = x.shape, wg.shape[0]
    e = 2.0 ** -23
    g, u = x @ wg.t(), x @ wu.t()
    a, da = act64(g, act)
    h, dh = a * u, dy @ wd
    dg, du = dh * u * da, dh * a
    eg, eu = D * e * (x.abs() @ wg.abs().t()), D * e * (x.abs() @ wu.abs().t())
    edh = D * e * (dy.abs() @ wd.abs())
    da1 = da.abs() + eg  # the second derivatives are below 1
    eh = (u.abs() + eu) * da1 * eg + a.abs() * eu + (ACT + R) * h.abs()
    edg = (u * da).abs() * edh + dh.abs() * (da1 * eu + u.abs() * eg) + (2 * ACT + R) * dg.abs() + ACT * (dh * u).abs()
    edu = a.abs() * edh + dh.abs() * da1 * eg + (ACT + R) * du.abs()
    out = {}

    def put(name, value, bound):
        out[name] = (value, bound * 1.01 + R * value.abs() + 1e-30)

    put("out", h @ wd.t(), (eh + F * e * h.abs()) @ wd.abs().t())
    put("dx", dg @ wg + du @ wu, (edg + 2 * F * e * dg.abs()) @ wg.abs() + (edu + 2 * F * e * du.abs()) @ wu.abs())
    put("dwg", dg.t() @ x, (edg + T * e * dg.abs()).t() @ x.abs())
    put("dwu", du.t() @ x, (edu + T * e * du.abs()).t() @ x.abs())
    put("dwd", dy.t() @ h, dy.abs().t() @ (eh + T * e * h.abs()))
    out["saved"] = (torch.stack([g, u]), torch.stack([eg, eu]) + 1e-30)
    return out


def inputs(T, D, F, seed, lead=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def make(r, c, std):
        big = torch.empty(lead + r * c, dtype=BF16, device=DEV)
        v = big[lead:].view(r, c)
        v.copy_(torch.randn(r, c, generator=gen, device=DEV) * std)
        return v
    return make(T, D, 1.0), make(F, D, D ** -0.5), make(F, D, D ** -0.5), make(D, F, F ** -0.5), make(T, D, 0.1)


def forward_backward(x, wg, wu, wd, dy, act, fill=5.0, **kw):
    (T, D), F = x.shape, wg.shape[0]
    saved = torch.full((2, T, F), fill, device=DEV)
    got = {"out": torch.full((T, D), fill, dtype=BF16, device=DEV), "dx": torch.full((T, D), fill, dtype=BF16, device=DEV),
           "dwg": torch.full((F, D), fill, dtype=BF16, device=DEV), "dwu": torch.full((F, D), fill, dtype=BF16, device=DEV),
           "dwd": torch.full((D, F), fill, dtype=BF16, device=DEV)}
    ccl.ccl_gated_ffn(x, wg, wu, wd, got["out"], act=act, saved=saved, **kw)
    ccl.ccl_gated_ffn_grad(dy, x, wg, wu, wd, saved, got["dx"], got["dwg"], got["dwu"], got["dwd"], act=act, **kw)
    got["saved"] = saved
    return got


def check(got, want):
    for name, t in got.items():
        value, bound = want[name]
        bad = ~((t.double() - value).abs() <= bound)
        assert not bool(bad.any()), "%s: %d of %d off, worst %g" % (
            name, int(bad.sum()), bad.numel(), float(((t.double() - value).abs() / bound).nan_to_num(9e9).max()))
    assert ccl.ccl_gated_ffn_timeouts() == 0


# one tile; ragged tiles; widths that pack; few tokens (split sums); several tiles each way
SHAPES = [(256, 64, 128), (1, 8, 8), (1, 512, 1024), (3, 200, 72), (8, 1024, 520), (9, 1024, 520), (37, 136, 1000), (130, 264, 1032), (257, 129, 255),
          (1, 1, 1), (5, 37, 41), (300, 1001, 333), (1000, 512, 776), (700, 1536, 2048)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,D,F", SHAPES)
def test_forward_and_backward(T, D, F, act):
    args = inputs(T, D, F, T + D + F)
    check(forward_backward(*args, act), reference(*args, act))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 7, 8, 15, 16, 17, 31, 33, 48, 64, 65, 128])
def test_few_tokens_without_saving(T):
    args = inputs(T, 768, 1088, T)
    out = torch.full((T, 768), 5.0, dtype=BF16, device=DEV)
    ccl.ccl_gated_ffn(*args[:4], out)
    check({"out": out}, {"out": reference(*args, "silu")["out"]})


# either side of each product's choice of tile: 64 and 128 tokens, 2^24 weights
@pytest.mark.parametrize("T,D,F", [(64, 260, 520), (65, 260, 520), (128, 260, 520), (129, 260, 520), (64, 2048, 8192), (65, 2048, 8191),
                                   (65, 2048, 8192), (128, 2048, 8192), (129, 2048, 8192)])
def test_forward_and_backward_where_the_tile_changes(T, D, F):
    args = inputs(T, D, F, T + D + F)
    check(forward_backward(*args, "silu"), reference(*args, "silu"))


@pytest.mark.parametrize("lead", [1, 4])
def test_buffers_with_their_elements_alignment_only(lead):
    args = inputs(70, 96, 136, lead, lead)
    check(forward_backward(*args, "silu"), reference(*args, "silu"))


def test_token_rows_do_not_depend_on_their_neighbours():
    """A row of NaN and a row of infinities leave the other rows' bits alone."""
    x, wg, wu, wd, dy = inputs(40, 128, 264, 3)
    clean = torch.empty(40, 128, dtype=BF16, device=DEV)
    ccl.ccl_gated_ffn(x, wg, wu, wd, clean)
    x[7], x[20] = math.nan, math.inf
    out = torch.empty_like(clean)
    ccl.ccl_gated_ffn(x, wg, wu, wd, out)
    rest = [i for i in range(40) if i not in (7, 20)]
    assert torch.equal(out[rest], clean[rest])
    assert bool(torch.isnan(out[7]).all()) and not bool(torch.isfinite(out[20]).any())


def test_accumulates_and_skips_gradients():
    args = inputs(90, 136, 264, 6)
    x, wg, wu, wd, dy = args
    want = reference(*args, "silu")
    got = forward_backward(*args, "silu")
    old = [torch.randn(264, 136, device=DEV).to(BF16), torch.randn(264, 136, device=DEV).to(BF16), torch.randn(136, 264, device=DEV).to(BF16)]
    acc = [t.clone() for t in old]
    dx = torch.empty_like(x)
    ccl.ccl_gated_ffn_grad(dy, x, wg, wu, wd, got["saved"], dx, *acc, accumulate=True)
    assert torch.equal(dx, got["dx"])
    for name, o, a in zip(("dwg", "dwu", "dwd"), old, acc):
        value, bound = want[name]
        total = o.double() + value
        assert bool(((a.double() - total).abs() <= bound + R * total.abs()).all())
    for k, name in enumerate(("dx", "dwg", "dwu", "dwd")):
        one = [None] * 4
        one[k] = torch.full_like(got[name], 3.0)
        ccl.ccl_gated_ffn_grad(dy, x, wg, wu, wd, got["saved"], *one)
        assert torch.equal(one[k], got[name])


def test_empty_sizes():
    e = lambda *s: torch.empty(*s, dtype=BF16, device=DEV)  # noqa: E731
    ccl.ccl_gated_ffn(e(0, 16), e(24, 16), e(24, 16), e(16, 24), e(0, 16))
    out = torch.full((5, 16), 2.0, dtype=BF16, device=DEV)
    ccl.ccl_gated_ffn(torch.ones(5, 16, dtype=BF16, device=DEV), e(0, 16), e(0, 16), e(16, 0), out)
    assert bool((out == 0).all())
    grads = [torch.full((24, 16), 2.0, dtype=BF16, device=DEV), torch.full((24, 16), 2.0, dtype=BF16, device=DEV), torch.full((16, 24), 2.0, dtype=BF16, device=DEV)]
    args = (e(0, 16), e(0, 16), e(24, 16), e(24, 16), e(16, 24), torch.empty(2, 0, 24, device=DEV), None)
    ccl.ccl_gated_ffn_grad(*args, *grads, accumulate=True)
    assert all(bool((g == 2).all()) for g in grads)
    ccl.ccl_gated_ffn_grad(*args, *grads)
    assert all(bool((g == 0).all()) for g in grads)


def test_gradient_against_differences():
    """<dy, out(w + h d) - out(w - h d)> / 2h against <grad, d>, the weights
    exactly representable.  Outputs are bf16: each is off by R |out| plus the
    rounding of h that the bound of `out` holds, and that over h is the
    tolerance, with the h^2 term of the third derivative (below 1)."""
    T, D, F, h = 64, 64, 128, 2.0 ** -2
    args = list(inputs(T, D, F, 9))
    want = reference(*args, "silu")
    got = forward_backward(*args, "silu")
    dy = args[4].double()
    for k, name in ((1, "dwg"), (2, "dwu"), (3, "dwd")):
        gen = torch.Generator(device=DEV).manual_seed(k)
        d = torch.randn(args[k].shape, generator=gen, device=DEV).sign() * 2.0 ** -5
        outs, slack, moved = [], 0.0, []
        for sign in (1, -1):
            w = list(args)
            w[k] = (args[k].float() + sign * h * d).to(BF16)
            moved.append(w[k].double())
            o = torch.empty(T, D, dtype=BF16, device=DEV)
            ccl.ccl_gated_ffn(*w[:4], o)
            outs.append(o.double())
            slack += float((dy.abs() * reference(*w, "silu")["out"][1]).pow(2).sum().sqrt())
        step = moved[0] - moved[1]  # what the weights really moved by
        quotient = float((dy * (outs[0] - outs[1])).sum())
        along = float((got[name].double() * step).sum())
        second = float((want[name][1] * step.abs()).pow(2).sum().sqrt())
        assert abs(quotient - along) <= 6 * (slack + second) + 0.05 * abs(along), name


def test_same_bits_each_time_in_a_graph_and_on_another_stream():
    args = inputs(100, 256, 512, 12)
    work = torch.empty(ccl.ccl_plan_gated_ffn_work_bytes(100, 256, 512, backward=True), dtype=torch.uint8, device=DEV)
    want = forward_backward(*args, "silu", work=work)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = forward_backward(*args, "silu", stream=s)  # its work buffers are allocated on s
    s.synchronize()
    for k in want:
        assert torch.equal(want[k], again[k]), k
    x, wg, wu, wd, dy = args
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ccl.ccl_gated_ffn(x, wg, wu, wd, out, saved=want["saved"], work=work)
    out.fill_(1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want["out"])
