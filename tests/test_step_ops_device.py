"""The training-step operators' binding on a machine with several GPUs, without
one: the C entries launch on the current device, so the binding makes the
tensors' device current for the call, takes that device's stream, and counts
the work buffer among the tensors that have to share it.  A stand-in for the
library records the device that is current when an entry is called."""
import contextlib

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl
from ring_allreduce_rank_gb300 import ccl as C

BF16 = torch.bfloat16


class Library:
    """Every entry succeeds and notes (name, current device, stream)."""

    def __init__(self, gpu):
        self.gpu, self.calls = gpu, []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, self.gpu["current"], args[-1]))
            return 0
        return entry


@pytest.fixture
def machine(monkeypatch):
    """Tensors on device `tensors`, with device 0 current."""
    gpu = {"current": 0, "tensors": 1, "seen": None}
    library = Library(gpu)

    @contextlib.contextmanager
    def device(d):
        was, gpu["current"] = gpu["current"], int(d)
        try:
            yield
        finally:
            gpu["current"] = was

    def on_gpu(*ts):
        gpu["seen"] = ts
        return gpu["tensors"]
    monkeypatch.setattr(C, "lib", lambda: library)
    monkeypatch.setattr(C, "_on_gpu", on_gpu)
    monkeypatch.setattr(C, "_raw_stream", lambda d: 1000 + d)
    monkeypatch.setattr(C, "_current_device", lambda: gpu["current"], raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: gpu["current"])
    monkeypatch.setattr(torch.cuda, "device", device)
    gpu["library"] = library
    return gpu


def _calls(work):
    n, d, f, v, k = 4, 8, 16, 20, 3
    m = lambda *s: torch.zeros(*s, dtype=BF16)  # noqa: E731
    ids, x, table = torch.zeros(n, dtype=torch.int64), m(n, d), m(v, d)
    wg, wu, wd, saved = m(f, d), m(f, d), m(d, f), torch.zeros(2, n, f)
    logits, tids, tl = m(n, v), torch.zeros(n, k, dtype=torch.int64), torch.zeros(n, k)
    loss, stats = torch.zeros(n), torch.zeros(n, 2)
    return {
        "ccl_embedding": lambda: ccl.ccl_embedding(table, ids, x),
        "ccl_embedding_grad": lambda: ccl.ccl_embedding_grad(x, ids, table, work=work),
        "ccl_gated_ffn": lambda: ccl.ccl_gated_ffn(x, wg, wu, wd, m(n, d), work=work),
        "ccl_gated_ffn_grad": lambda: ccl.ccl_gated_ffn_grad(x, x, wg, wu, wd, saved, m(n, d), work=work),
        "ccl_distill_loss": lambda: ccl.ccl_distill_loss(logits, tids, tl, loss),
        "ccl_distill_grad": lambda: ccl.ccl_distill_grad(logits, tids, tl, stats, m(n, v)),
    }


OPERATORS = list(_calls(None))
WORKING = ["ccl_embedding_grad", "ccl_gated_ffn", "ccl_gated_ffn_grad"]


@pytest.mark.parametrize("tensors", [0, 1])
@pytest.mark.parametrize("name", OPERATORS)
def test_the_tensors_device_is_current_during_the_call(machine, name, tensors):
    machine["tensors"] = tensors
    _calls(torch.zeros(1 << 20, dtype=torch.uint8))[name]()
    assert machine["library"].calls == [(name, tensors, 1000 + tensors)]
    assert machine["current"] == 0  # as it was


@pytest.mark.parametrize("name", WORKING)
def test_the_work_buffer_is_among_the_tensors_that_share_a_device(machine, name):
    work = torch.zeros(1 << 20, dtype=torch.uint8)
    _calls(work)[name]()
    assert any(t is work for t in machine["seen"])


def test_tensors_on_two_devices_are_refused():
    class On:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device
    assert C._on_gpu(On(1), None, On(1)) == 1
    with pytest.raises(ValueError, match="different devices"):
        C._on_gpu(On(1), On(0))
    with pytest.raises(ValueError, match="CUDA"):
        C._on_gpu(On(1), On(-1))
    with pytest.raises(ValueError, match="CUDA"):
        C._on_gpu(On(-1), On(1))
    with pytest.raises(ValueError, match="CUDA"):
        ccl.ccl_embedding(None, None, None)
