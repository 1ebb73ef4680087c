"""ccl_expert_ffn and ccl_expert_ffn_grad against the formulas in 64 bits, expert
by expert.

Bounds, with r = 2^-8 (bf16's unit roundoff): an fp32 sum of n products is good to
n 2^-23 of the sum of magnitudes, an activation to 2^-18 of itself; h, dg and du
carry those errors of their factors and one rounding r, which the next product
sums; each output is rounded once more.  The backward pass starts from the g, u
and x that the 8 bits hold, which are exact numbers: the gradients are compared
with those of these numbers, and the numbers with g, u and x by half a step."""
import math

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F64, I32 = torch.bfloat16, torch.float64, torch.int32
R = 2.0 ** -8
ACT = 2.0 ** -18
E = 2.0 ** -23


def act64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


def offsets_of(counts, start=0):
    return torch.tensor([start], device=DEV).repeat(len(counts) + 1).add_(torch.tensor([0] + list(counts), device=DEV).cumsum(0)).to(I32)


def inputs(counts, D, F, seed, lead=0, start=0, behind=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, rows = len(counts), start + sum(counts) + behind

    def make(std, *shape):
        big = torch.empty(lead + math.prod(shape), dtype=BF16, device=DEV)
        v = big[lead:].view(shape)
        v.copy_(torch.randn(*shape, generator=g, device=DEV) * std)
        return v
    return {"x": make(1.0, rows, D), "offsets": offsets_of(counts, start), "wg": make(D ** -0.5, n, F, D), "wu": make(D ** -0.5, n, F, D),
            "wd": make(F ** -0.5, n, D, F), "dy": make(0.1, rows, D)}


def saved_of(rows, F, fill=0):
    w = ccl.ccl_plan_act8_width(F)
    return (torch.full((2, rows, w), fill, dtype=torch.int8, device=DEV), torch.full((2, rows, w // 32), fill, dtype=torch.uint8, device=DEV))


def values_of(saved, F):
    codes, scales = saved
    step = ((scales.to(torch.int64) - 127 + 1023) << 52).view(F64)  # 2^e, exactly
    return (codes.to(F64) * step.repeat_interleave(32, dim=-1))[..., :F], step.repeat_interleave(32, dim=-1)[..., :F]


def act8_of(x):
    w = ccl.ccl_plan_act8_width(x.shape[1])
    out = (torch.empty(x.shape[0], w, dtype=torch.int8, device=DEV), torch.empty(x.shape[0], w // 32, dtype=torch.uint8, device=DEV))
    ccl.ccl_act8_pack(x, *out)
    return out


def forward(a, act="silu", saved=None, fill=5.0, **kw):
    out = torch.full(a["x"].shape, fill, dtype=BF16, device=DEV)
    ccl.ccl_expert_ffn(a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], out, act=act, saved=saved, **kw)
    return out


def backward(a, saved, act="silu", x=None, fill=5.0, old=None, **kw):
    got = {"dx": torch.full(a["x"].shape, fill, dtype=BF16, device=DEV)}
    for k in ("wg", "wu", "wd"):
        got["d" + k] = torch.full(a[k].shape, fill, dtype=BF16, device=DEV) if old is None else old["d" + k].clone()
    ccl.ccl_expert_ffn_grad(a["dy"], a["x"] if x is None else x, a["offsets"], a["wg"], a["wu"], a["wd"], saved, got["dx"], got["dwg"], got["dwu"],
                            got["dwd"], act=act, accumulate=old is not None, **kw)
    return got


def spans(a):
    o = a["offsets"].tolist()
    return [slice(o[e], o[e + 1]) for e in range(len(o) - 1)]


def check(name, got, value, bound):
    bad = ~((got.to(F64) - value).abs() <= bound * 1.01 + R * value.abs() + 1e-30)
    assert not bool(bad.any()), "%s: %d of %d off, worst %g" % (name, int(bad.sum()), bad.numel(), float(((got.to(F64) - value).abs() / (bound + R * value.abs() + 1e-30)).nan_to_num(9e9).max()))


def check_forward(a, out, act, saved=None):
    for e, s in enumerate(spans(a)):
        x, wg, wu, wd = (t.to(F64) for t in (a["x"][s], a["wg"][e], a["wu"][e], a["wd"][e]))
        D, F = x.shape[1], wg.shape[0]
        g, u = x @ wg.T, x @ wu.T
        av, da = act64(g, act)
        h = av * u
        eg, eu = D * E * (x.abs() @ wg.abs().T), D * E * (x.abs() @ wu.abs().T)
        eh = (u.abs() + eu) * (da.abs() + eg) * eg + av.abs() * eu + (ACT + R) * h.abs()
        check("out of expert %d" % e, out[s], h @ wd.T, (eh + F * E * h.abs()) @ wd.abs().T)
        if saved is not None:
            v, step = values_of(saved, F)
            for k, (t, err) in enumerate(((g, eg), (u, eu))):
                assert bool(((v[k][s] - t).abs() <= step[k][s] / 2 * 1.0001 + err + 1e-30).all())
                if t.numel():  # the step is below twice the least that would do
                    assert bool((step[k][s] <= 2 / 127 * (t.abs() + err).amax() + 2.0 ** -126).all())
    left = torch.ones(out.shape[0], dtype=torch.bool, device=DEV)
    left[spans(a)[0].start:spans(a)[-1].stop] = False
    assert bool((out[left] == 5).all())  # rows of no expert are left as they were
    assert ccl.ccl_gated_ffn_timeouts() == 0


def check_backward(a, got, saved, act, x8=None, old=None):
    for e, s in enumerate(spans(a)):
        x = (a["x"] if x8 is None else values_of(x8, a["x"].shape[1])[0])[s].to(F64)
        dy, wg, wu, wd = (t.to(F64) for t in (a["dy"][s], a["wg"][e], a["wu"][e], a["wd"][e]))
        (T, D), F = x.shape, wg.shape[0]
        v = values_of(saved, F)[0]
        g, u = v[0][s], v[1][s]
        av, da = act64(g, act)
        h, dh = av * u, dy @ wd
        dg, du = dh * u * da, dh * av
        edh = D * E * (dy.abs() @ wd.abs())
        eh = (ACT + R) * h.abs()
        edg = (u * da).abs() * edh + (2 * ACT + R) * dg.abs() + ACT * (dh * u).abs()
        edu = av.abs() * edh + (ACT + R) * du.abs()
        if got["dx"] is not None:
            check("dx of expert %d" % e, got["dx"][s], dg @ wg + du @ wu, (edg + 2 * F * E * dg.abs()) @ wg.abs() + (edu + 2 * F * E * du.abs()) @ wu.abs())
        for name, value, bound in (("dwg", dg.T @ x, (edg + T * E * dg.abs()).T @ x.abs()), ("dwu", du.T @ x, (edu + T * E * du.abs()).T @ x.abs()),
                                   ("dwd", dy.T @ h, dy.abs().T @ (eh + T * E * h.abs()))):
            if old is not None:
                value = value + old[name][e].to(F64)
            check("%s of expert %d" % (name, e), got[name][e], value, bound)
    left = torch.ones(got["dx"].shape[0], dtype=torch.bool, device=DEV)
    left[spans(a)[0].start:spans(a)[-1].stop] = False
    assert bool((got["dx"][left] == 5).all())
    assert ccl.ccl_gated_ffn_timeouts() == 0


# rows of each expert, dim, ffn.  One row; experts without rows; ragged tiles; more rows than a tile; odd widths; both kernels of the forward pass
# (an average of 64 rows lies between them), with and without sums cut along K, several tiles of few tokens, and large weights
CASES = [([1], 8, 8), ([2], 64, 128), ([0, 1, 0, 1], 512, 1024), ([3, 0, 5, 1], 200, 72), ([7, 130, 0, 33], 136, 264), ([64, 64], 64, 32), ([63, 65, 1, 128], 96, 160),
         ([200], 264, 1032), ([257, 0, 300, 511], 256, 512), ([5, 4], 37, 41), ([100, 301, 0], 129, 255), ([1, 2, 3, 4, 5, 6, 7, 8], 1001, 333), ([1] * 40, 72, 136),
         ([1000, 24], 512, 776), ([300, 700], 1536, 1000), ([16, 16, 200], 768, 1088), ([0, 0, 520], 1, 1),
         ([100] + [1] * 39, 72, 136), ([50, 70], 2048, 8192), ([30, 33], 2048, 8191)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,D,F", CASES)
def test_forward_and_backward(counts, D, F, act):
    a = inputs(counts, D, F, D + F, behind=3)
    saved = saved_of(a["x"].shape[0], F)
    out = forward(a, act, saved)
    check_forward(a, out, act, saved)
    assert torch.equal(forward(a, act), out)  # keeping g and u changes nothing
    check_backward(a, backward(a, saved, act), saved, act)
    x8 = act8_of(a["x"])
    check_backward(a, backward(a, saved, act, x=x8), saved, act, x8)


@pytest.mark.parametrize("T", [1, 2, 8, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_rows_of_one_expert_among_empty_ones(T):
    a = inputs([0, T, 0, 0], 328, 584, T, start=2, behind=1)
    saved = saved_of(a["x"].shape[0], 584)
    check_forward(a, forward(a, saved=saved), "silu", saved)
    check_backward(a, backward(a, saved), saved, "silu")


def test_many_experts():
    counts = [(7 * e) % 4 for e in range(1024)]
    a = inputs(counts, 40, 72, 1)
    saved = saved_of(a["x"].shape[0], 72)
    check_forward(a, forward(a, saved=saved), "silu", saved)
    check_backward(a, backward(a, saved), saved, "silu")


@pytest.mark.parametrize("lead", [1, 4])
def test_buffers_with_their_elements_alignment_only(lead):
    for counts in ([5, 30], [200, 100]):
        a = inputs(counts, 96, 136, lead, lead)
        saved = saved_of(a["x"].shape[0], 136)
        check_forward(a, forward(a, saved=saved), "silu", saved)
        check_backward(a, backward(a, saved), saved, "silu")


@pytest.mark.parametrize("counts", [[20, 12, 9], [150, 70, 90]])
def test_experts_and_rows_do_not_meet(counts):
    """NaN and infinities in one expert's weights, in one row, and behind the last
    expert leave every other row's and expert's results alone."""
    a = inputs(counts, 136, 264, 3, start=4, behind=70)
    saved = saved_of(a["x"].shape[0], 264)
    clean, grads = forward(a, saved=saved), None
    grads = backward(a, saved)
    b = {k: v.clone() for k, v in a.items()}
    b["wg"][1, 0], b["wd"][1, 3] = math.nan, math.inf
    end = 4 + sum(counts)
    b["x"][end:], b["dy"][end:], b["x"][:4], b["dy"][:4] = math.nan, math.nan, math.inf, math.inf
    b["x"][4], b["dy"][4] = math.nan, math.nan
    saved2 = saved_of(a["x"].shape[0], 264, 7)
    saved2[1][:, end:] = 255
    out = forward(b, saved=saved2)
    first, second, third = spans(a)
    keep = list(range(first.start + 1, first.stop)) + list(range(third.start, third.stop))
    assert torch.equal(out[keep], clean[keep]) and bool(torch.isnan(out[4]).all()) and not bool(torch.isfinite(out[second]).any())
    got = backward(b, saved2)
    assert torch.equal(got["dx"][keep], grads["dx"][keep])
    for k in ("dwg", "dwu", "dwd"):
        assert torch.equal(got[k][2], grads[k][2]) and bool(torch.isnan(got[k][0]).all())


def test_offsets_that_fall_or_lie_outside():
    """Taken as the largest before them within the rows."""
    a = inputs([3, 4, 5, 6], 64, 96, 4)
    n = a["x"].shape[0]
    for wild, tame in (([0, 9, 4, 12, 18], [0, 9, 9, 12, 18]), ([-5, 2, 2 ** 31 - 1, 3, 18], [0, 2, n, n, n]), ([n, 0, n, 0, n], [n, n, n, n, n]),
                       ([0, n, 0, n, 0], [0, n, n, n, n])):
        saved, same = saved_of(n, 96), saved_of(n, 96)
        outs, grads = [], []
        for o, s in ((wild, saved), (tame, same)):
            b = dict(a, offsets=torch.tensor(o, device=DEV).to(I32))
            outs.append(forward(b, saved=s))
            grads.append(backward(b, s))
        assert torch.equal(*outs) and torch.equal(saved[0], same[0])
        assert all(torch.equal(grads[0][k], grads[1][k]) for k in grads[0])


def test_accumulates_and_skips_gradients():
    for counts in ([90, 0, 33], [600, 0, 1]):
        a = inputs(counts, 136, 264, 6)
        saved = saved_of(a["x"].shape[0], 264)
        forward(a, saved=saved)
        got = backward(a, saved)
        old = {"d" + k: torch.randn(a[k].shape, device=DEV).to(BF16) for k in ("wg", "wu", "wd")}
        more = backward(a, saved, old=old)
        check_backward(a, more, saved, "silu", old=old)
        for k in old:
            assert torch.equal(more[k][1], old[k][1]) and bool((got[k][1] == 0).all())  # an expert without rows
        for k, name in enumerate(("dx", "dwg", "dwu", "dwd")):
            one = [None] * 4
            one[k] = torch.full_like(got[name], 5.0)
            ccl.ccl_expert_ffn_grad(a["dy"], a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], saved, *one)
            assert torch.equal(one[k], got[name])


@pytest.mark.parametrize("counts,D,F,lead", [([90, 0, 33], 37, 41, 0), ([600, 0, 1], 129, 255, 0), ([65, 0, 130], 301, 96, 1), ([40, 0, 70], 264, 129, 0),
                                             ([10, 0, 300], 136, 264, 3), ([80, 0, 5], 1, 1, 0)])
def test_accumulates_in_odd_rows(counts, D, F, lead):
    a = inputs(counts, D, F, 8, lead=lead)
    saved = saved_of(a["x"].shape[0], F)
    forward(a, saved=saved)
    old = {"d" + k: torch.randn(a[k].shape, device=DEV).to(BF16) for k in ("wg", "wu", "wd")}
    more = backward(a, saved, old=old)
    check_backward(a, more, saved, "silu", old=old)
    for k in old:
        assert torch.equal(more[k][1], old[k][1])  # an expert without rows


def test_no_rows():
    e = lambda *s: torch.empty(*s, dtype=BF16, device=DEV)  # noqa: E731
    o = torch.zeros(4, device=DEV, dtype=I32)
    ccl.ccl_expert_ffn(e(0, 16), o, e(3, 24, 16), e(3, 24, 16), e(3, 16, 24), e(0, 16), saved=saved_of(0, 24))
    grads = [torch.full(s, 2.0, dtype=BF16, device=DEV) for s in ((3, 24, 16), (3, 24, 16), (3, 16, 24))]
    args = (e(0, 16), e(0, 16), o, e(3, 24, 16), e(3, 24, 16), e(3, 16, 24), saved_of(0, 24), None)
    ccl.ccl_expert_ffn_grad(*args, *grads, accumulate=True)
    assert all(bool((g == 2).all()) for g in grads)
    ccl.ccl_expert_ffn_grad(*args, *grads)
    assert all(bool((g == 0).all()) for g in grads)
    for n in (5, 500):  # rows, but none of an expert's
        out = torch.full((n, 16), 5.0, dtype=BF16, device=DEV)
        x = torch.ones(n, 16, dtype=BF16, device=DEV)
        ccl.ccl_expert_ffn(x, o, e(3, 24, 16), e(3, 24, 16), e(3, 16, 24), out)
        assert bool((out == 5).all())
        grads = [torch.full(s, 2.0, dtype=BF16, device=DEV) for s in ((3, 24, 16), (3, 24, 16), (3, 16, 24))]
        ccl.ccl_expert_ffn_grad(x, x, o, e(3, 24, 16), e(3, 24, 16), e(3, 16, 24), saved_of(n, 24), out, *grads)
        assert bool((out == 5).all()) and all(bool((g == 0).all()) for g in grads)


def test_one_expert_is_the_dense_block():
    """The forward pass of one expert agrees with ccl_gated_ffn to the roundings of
    both."""
    a = inputs([300], 264, 520, 8)
    out, dense = forward(a), torch.empty(300, 264, dtype=BF16, device=DEV)
    ccl.ccl_gated_ffn(a["x"], a["wg"][0], a["wu"][0], a["wd"][0], dense)
    check_forward(a, out, "silu")
    check_forward(a, dense, "silu")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """Of the function that the 8 bits keep, in 64 bits: y(g, u) = (act(g) u) wd^T
    differentiated along random directions of x, through g = x wg^T and u = x wu^T
    moved from the kept g and u.  Central differences with h = 2^-10: their error is
    h^2 times a third derivative along the direction, the gradient's its bound."""
    a = inputs([40, 24], 64, 96, 9)
    n, h = 64, 2.0 ** -10
    saved = saved_of(n, 96)
    forward(a, act, saved)
    got = backward(a, saved, act)
    v = values_of(saved, 96)[0]
    gen = torch.Generator(device=DEV).manual_seed(2)
    for _ in range(5):
        d = torch.randn(n, 64, generator=gen, device=DEV, dtype=F64)
        quotient, along, slack = 0.0, 0.0, 0.0
        for e, s in enumerate(spans(a)):
            dy, wg, wu, wd = (t.to(F64) for t in (a["dy"][s], a["wg"][e], a["wu"][e], a["wd"][e]))
            sides = []
            for sign in (1, -1):
                g, u = v[0][s] + sign * h * d[s] @ wg.T, v[1][s] + sign * h * d[s] @ wu.T
                sides.append(((act64(g, act)[0] * u) @ wd.T * dy).sum())
            quotient += float(sides[0] - sides[1]) / (2 * h)
            along += float((got["dx"][s].to(F64) * d[s]).sum())
            # each entry of dx is off by a few r of the size of what it sums; these errors are independent of d
            dh = dy @ wd
            size = (dh.abs() * v[1][s].abs() * 1.2) @ wg.abs() + (dh.abs() * act64(v[0][s], act)[0].abs()) @ wu.abs()
            slack += float(((2 * R * size * d[s]) ** 2).sum())
        assert abs(quotient - along) <= 4 * math.sqrt(slack) + 1e3 * h * h


def test_same_bits_each_time_in_a_graph_and_on_another_stream():
    for counts in ([20, 0, 41], [200, 0, 341]):
        a = inputs(counts, 256, 512, 12)
        n = a["x"].shape[0]
        work = torch.empty(ccl.ccl_plan_expert_ffn_work_bytes(n, 3, 256, 512, backward=True), dtype=torch.uint8, device=DEV)
        saved = saved_of(n, 512)
        out = forward(a, saved=saved, work=work)
        want = backward(a, saved, work=work)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            saved2 = saved_of(n, 512)
            out2 = forward(a, saved=saved2, stream=s)
            got = backward(a, saved2, stream=s)
        s.synchronize()
        assert torch.equal(out, out2) and torch.equal(saved[0], saved2[0]) and all(torch.equal(want[k], got[k]) for k in want)
        g = torch.cuda.CUDAGraph()
        out3, saved3, grads = torch.zeros_like(out), saved_of(n, 512), {k: torch.zeros_like(v) for k, v in want.items()}
        with torch.cuda.graph(g):
            ccl.ccl_expert_ffn(a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], out3, saved=saved3, work=work)
            ccl.ccl_expert_ffn_grad(a["dy"], a["x"], a["offsets"], a["wg"], a["wu"], a["wd"], saved3, grads["dx"], grads["dwg"], grads["dwu"],
                                    grads["dwd"], work=work)
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, out3) and all(torch.equal(want[k], grads[k]) for k in want)
        # other counts in the same graph: nothing of them was kept on the host
        other = [sum(counts) - 11, 5, 6]
        a["offsets"].copy_(offsets_of(other))
        g.replay()
        torch.cuda.synchronize()
        check_forward(a, out3, "silu", saved3)
        check_backward(a, {k: v for k, v in grads.items()}, saved3, "silu")
