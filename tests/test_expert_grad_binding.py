"""ccl_expert_ffn_grad's binding where x or saved is left out, without a GPU: x is
needed for the gradients of w_gate and w_up only, saved always, and what is missing is
named."""
import pytest
import torch

import ring_allreduce_rank_gb300 as ccl
from test_step_ops_device import machine  # noqa: F401

BF16, I32 = torch.bfloat16, torch.int32
N, D, F, E = 4, 8, 16, 3


def _m(*s):
    return torch.zeros(*s, dtype=BF16)


def _call(x, saved, *grads, n=N):
    ccl.ccl_expert_ffn_grad(_m(n, D), x, torch.zeros(E + 1, dtype=I32), _m(E, F, D), _m(E, F, D), _m(E, D, F), saved, *grads,
                            work=torch.zeros(1 << 16, dtype=torch.uint8))


def _saved(n=N):
    return torch.zeros(2, n, 32, dtype=torch.int8), torch.zeros(2, n, 1, dtype=torch.uint8)


def _passed(machine, monkeypatch):
    """The arguments of the entry's calls."""
    calls = []
    monkeypatch.setattr(type(machine["library"]), "__getattr__", lambda self, name: lambda *args: calls.append((name, args)) or 0)
    return calls


@pytest.mark.parametrize("which", ["grad_x", "grad_w_down"])
@pytest.mark.parametrize("device", [0, 1])
def test_x_may_be_left_out_where_it_is_not_read(machine, monkeypatch, which, device):  # noqa: F811
    machine["tensors"] = device
    calls = _passed(machine, monkeypatch)
    grads = (_m(N, D),) if which == "grad_x" else (None, None, None, _m(E, D, F))
    _call(None, _saved(), *grads)
    (name, args), = calls
    assert name == "ccl_expert_ffn_grad" and args[1:4] == (None, None, None)
    assert [p is not None for p in args[17:21]] == [which == "grad_x", False, False, which == "grad_w_down"]


@pytest.mark.parametrize("k", [1, 2])
def test_x_is_asked_for_by_name(machine, k):  # noqa: F811
    grads = [None] * 4
    grads[k] = _m(E, F, D)
    with pytest.raises(ValueError, match="x is needed"):
        _call(None, _saved(), *grads)
    assert machine["library"].calls == []
    with pytest.raises(ValueError, match="x must be"):  # neither a tensor nor a pair
        _call((_m(N, D),), _saved(), *grads)


def test_saved_is_asked_for_by_name(machine):  # noqa: F811
    with pytest.raises(ValueError, match="saved is needed"):
        _call(_m(N, D), None, _m(N, D))
    with pytest.raises(ValueError, match="saved must be"):
        _call(_m(N, D), _saved()[:1], _m(N, D))
    with pytest.raises(ValueError, match="saved must be"):
        ccl.ccl_expert_ffn(_m(N, D), torch.zeros(E + 1, dtype=I32), _m(E, F, D), _m(E, F, D), _m(E, D, F), _m(N, D), saved=_saved()[:1])
    assert machine["library"].calls == []


def test_what_is_given_is_passed_as_before(machine, monkeypatch):  # noqa: F811
    calls = _passed(machine, monkeypatch)
    x, x8, saved = _m(N, D), (torch.zeros(N, 32, dtype=torch.int8), torch.zeros(N, 1, dtype=torch.uint8)), _saved()
    _call(x, saved, _m(N, D), _m(E, F, D))
    _call(x8, saved, _m(N, D), _m(E, F, D))
    assert calls[0][1][1:4] == (x.data_ptr(), None, None)
    assert calls[1][1][1:4] == (None, x8[0].data_ptr(), x8[1].data_ptr())
    for _, args in calls:
        assert args[8:10] == (saved[0].data_ptr(), saved[1].data_ptr())


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [136, 37])
def test_gradients_without_x_are_the_same(dim):
    from test_gpu_expert_ffn import backward, forward, inputs, saved_of
    a = inputs([90, 0, 33], dim, 264, 6)
    saved = saved_of(a["x"].shape[0], 264)
    forward(a, saved=saved)
    want = backward(a, saved)
    dx, dwd = torch.empty_like(want["dx"]), torch.empty_like(want["dwd"])
    ccl.ccl_expert_ffn_grad(a["dy"], None, a["offsets"], a["wg"], a["wu"], a["wd"], saved, dx, None, None, dwd)
    assert torch.equal(dx, want["dx"]) and torch.equal(dwd, want["dwd"])
