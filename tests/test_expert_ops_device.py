"""The expert-parallel operators' binding on a machine with several GPUs, without
one: every entry runs with the tensors' device current and on that device's
stream, and the work buffer and the 8-bit tensors count among the tensors that
have to share it."""
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl
from test_step_ops_device import machine  # noqa: F401

BF16, I32 = torch.bfloat16, torch.int32


def _calls(work):
    n, d, f, e, k = 4, 8, 16, 3, 2
    m = lambda *s: torch.zeros(*s, dtype=BF16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=I32)  # noqa: E731
    z, x, rows = torch.zeros(n, e), m(n, d), m(n * k, d)
    wg, wu, wd = m(e, f, d), m(e, f, d), m(e, d, f)
    c8 = lambda *s: (torch.zeros(*s, 32, dtype=torch.int8), torch.zeros(*s, 1, dtype=torch.uint8))  # noqa: E731
    x8, saved = c8(n), c8(2, n)
    t = {"x8": x8, "saved": saved}
    return t, {
        "ccl_route": lambda: ccl.ccl_route(z, i(n, k), torch.zeros(n, k), torch.zeros(n), i(e + 1), torch.zeros(e), torch.zeros(e), torch.zeros(2), work=work),
        "ccl_route_grad": lambda: ccl.ccl_route_grad(z, i(n, k), torch.zeros(n), i(e + 1), torch.zeros(e), torch.zeros(n, k), z),
        "ccl_expert_order": lambda: ccl.ccl_expert_order(i(n, k), i(e + 1), i(n, k), work=work),
        "ccl_dispatch": lambda: ccl.ccl_dispatch(x, i(n, k), rows),
        "ccl_combine": lambda: ccl.ccl_combine(rows, i(n, k), x),
        "ccl_combine_grad": lambda: ccl.ccl_combine_grad(x, i(n, k), rows=rows, grad_weights=torch.zeros(n, k)),
        "ccl_act8_pack": lambda: ccl.ccl_act8_pack(x, *x8),
        "ccl_act8_unpack": lambda: ccl.ccl_act8_unpack(*x8, x),
        "ccl_expert_ffn": lambda: ccl.ccl_expert_ffn(x, i(e + 1), wg, wu, wd, m(n, d), saved=saved, work=work),
        "ccl_expert_ffn_grad": lambda: ccl.ccl_expert_ffn_grad(x, x8, i(e + 1), wg, wu, wd, saved, m(n, d), work=work),
    }


OPERATORS = list(_calls(None)[1])
WORKING = ["ccl_route", "ccl_expert_order", "ccl_expert_ffn", "ccl_expert_ffn_grad"]


@pytest.mark.parametrize("tensors", [0, 1])
@pytest.mark.parametrize("name", OPERATORS)
def test_the_tensors_device_is_current_during_the_call(machine, name, tensors):  # noqa: F811
    machine["tensors"] = tensors
    _calls(torch.zeros(1 << 20, dtype=torch.uint8))[1][name]()
    assert machine["library"].calls == [(name, tensors, 1000 + tensors)]
    assert machine["current"] == 0  # as it was


@pytest.mark.parametrize("name", WORKING)
def test_the_work_buffer_is_among_the_tensors_that_share_a_device(machine, name):  # noqa: F811
    work = torch.zeros(1 << 20, dtype=torch.uint8)
    _calls(work)[1][name]()
    assert any(t is work for t in machine["seen"])


@pytest.mark.parametrize("name,of", [("ccl_expert_ffn", "saved"), ("ccl_expert_ffn_grad", "saved"), ("ccl_expert_ffn_grad", "x8"), ("ccl_act8_pack", "x8")])
def test_the_8_bit_tensors_are_too(machine, name, of):  # noqa: F811
    tensors, calls = _calls(torch.zeros(1 << 20, dtype=torch.uint8))
    calls[name]()
    assert all(any(t is s for s in machine["seen"]) for t in tensors[of])
