"""The feed-forward block's gradients against central differences of its own
outputs, along the directions in which they are largest, so that a lost term, a
zero or a wrong sign is many times the tolerance.

For weights or inputs v and a step s along sign(gradient) (as bf16 holds it),
Q = <dy, out(v + s/2) - out(v - s/2)> against <grad, s>.  The tolerance is what
the two may differ by: each output's bound times |dy|, each gradient's bound
times |s|, and the difference quotient's own error, taken in 64 bits from
autograd, which shares no formula with the kernels."""
import importlib.util
import os

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl

_spec = importlib.util.spec_from_file_location("gated_ffn_bounds", os.path.join(os.path.dirname(os.path.abspath(__file__)), "test_gpu_gated_ffn.py"))
base = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(base)

pytestmark = pytest.mark.gpu
NAMES = ("dx", "dwg", "dwu", "dwd")


def exact(args, act):
    """The block in 64 bits and, by autograd, <dy, out>'s gradients."""
    x, wg, wu, wd = (t.double().requires_grad_() for t in args[:4])
    g = x @ wg.t()
    a = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    out = (a * (x @ wu.t())) @ wd.t()
    return out.detach(), torch.autograd.grad(out, (x, wg, wu, wd), args[4].double())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,D,F", [(64, 64, 128), (150, 72, 120), (33, 61, 77)])
def test_gradients_follow_the_outputs(T, D, F, act):
    args = list(base.inputs(T, D, F, 9))
    want = base.reference(*args, act)
    got = base.forward_backward(*args, act)
    dy = args[4].double()
    _, grads = exact(args, act)
    for k, name in enumerate(NAMES):
        size = 2.0 ** -4 if name == "dx" else 2.0 ** -7
        moved, outs, outs64, slack = [], [], [], 0.0
        for sign in (1, -1):
            v = list(args)
            v[k] = (args[k].double() + sign * size * grads[k].sign()).to(base.BF16)
            moved.append(v[k].double())
            out = torch.empty(T, D, dtype=base.BF16, device=args[0].device)
            ccl.ccl_gated_ffn(*v[:4], out, act=act)
            outs.append(out.double())
            outs64.append(exact(v, act)[0])
            slack += float((dy.abs() * base.reference(*v, act)["out"][1]).sum())
        step = moved[0] - moved[1]
        quotient, quotient64 = (float((dy * (o[0] - o[1])).sum()) for o in (outs, outs64))
        along, along64 = float((got[name].double() * step).sum()), float((grads[k] * step).sum())
        tolerance = slack + float((want[name][1] * step.abs()).sum()) + abs(quotient64 - along64)
        assert abs(quotient - along) <= tolerance, name
        # what the check is worth: neither no gradient nor its negative would pass
        assert abs(quotient) > 2 * tolerance and abs(quotient + along) > 2 * tolerance, (name, quotient, tolerance)
