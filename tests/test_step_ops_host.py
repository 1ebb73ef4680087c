"""The training-step operators' argument checks, without a GPU: the C entries
reject bad calls before anything is launched, the planners agree with the
documented layouts, and the binding names what is wrong with a tensor.  The C
calls run in a child process that sees no GPU, on fake pointers that are never
dereferenced."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import ring_allreduce_rank_gb300 as ccl
from ring_allreduce_rank_gb300 import ccl as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, OVERLAP = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ring_allreduce_rank_gb300 import build
    build.build()
    ccl.lib()


def _embedding(L, table=1 << 40, rows=10, dim=8, ts=8, dt=0, ids=2 << 40, n=4, first=0, out=3 << 40, os_=8):
    return L.ccl_embedding(table, rows, dim, ts, dt, ids, n, first, 1.0, out, os_, None)


def _embedding_grad(L, dy=1 << 40, ys=8, ids=2 << 40, n=4, rows=10, dim=8, dt=0, acc=0, grad=3 << 40, gs=8, work=4 << 40, nbytes=1 << 20):
    return L.ccl_embedding_grad(dy, ys, ids, n, 0, rows, dim, dt, 1.0, acc, grad, gs, work, nbytes, None)


def _ffn(L, x=1 << 40, wg=2 << 40, wu=3 << 40, wd=4 << 40, n=4, d=16, f=24, dt=1, act=0, out=5 << 40, saved=None, work=6 << 40, nbytes=1 << 26):
    return L.ccl_gated_ffn(x, wg, wu, wd, n, d, f, dt, act, out, saved, work, nbytes, None)


def _ffn_grad(L, dy=8 << 40, x=1 << 40, wg=2 << 40, wu=3 << 40, wd=4 << 40, saved=5 << 40, n=4, d=16, f=24, dt=1, act=0, acc=0, dx=9 << 40,
              dwg=10 << 40, dwu=11 << 40, dwd=12 << 40, work=6 << 40, nbytes=1 << 26):
    return L.ccl_gated_ffn_grad(dy, x, wg, wu, wd, saved, n, d, f, dt, act, acc, dx, dwg, dwu, dwd, work, nbytes, None)


def _distill(L, logits=1 << 40, n=4, v=100, ls=100, dt=0, ids=2 << 40, t=3 << 40, top=5, tau=1.0, w=None, loss=4 << 40, stats=None, grad=None, gs=100):
    return L.ccl_distill_loss(logits, n, v, ls, dt, ids, t, top, tau, w, loss, stats, grad, gs, None)


def _distill_grad(L, logits=1 << 40, n=4, v=100, ls=100, dt=0, ids=2 << 40, t=3 << 40, top=5, tau=1.0, w=None, stats=4 << 40, grad=5 << 40, gs=100):
    return L.ccl_distill_grad(logits, n, v, ls, dt, ids, t, top, tau, w, stats, grad, gs, None)


def refusals(L):
    for kw in (dict(dt=5), dict(ts=7), dict(os_=7), dict(table=None), dict(ids=None), dict(out=None), dict(rows=1 << 31), dict(n=1 << 31),
               dict(dim=(1 << 24) + 1, ts=1 << 25, os_=1 << 25), dict(ts=1 << 62)):
        assert _embedding(L, **kw) == INVALID, kw
    assert _embedding(L, out=(1 << 40) + 16) == OVERLAP
    assert _embedding(L, out=(2 << 40) + 8) == OVERLAP
    assert _embedding(L, n=0, ids=None, out=None) == 0
    for kw in (dict(dt=9), dict(ys=7), dict(gs=7), dict(dy=None), dict(ids=None), dict(grad=None), dict(work=None), dict(nbytes=16), dict(work=(4 << 40) + 8),
               dict(rows=1 << 31), dict(n=1 << 31), dict(gs=1 << 62)):
        assert _embedding_grad(L, **kw) == INVALID, kw
    assert _embedding_grad(L, grad=(1 << 40) + 32) == OVERLAP
    assert _embedding_grad(L, work=(3 << 40)) == OVERLAP
    assert _embedding_grad(L, rows=0) == 0
    assert _embedding_grad(L, n=0, acc=1) == 0
    for kw in (dict(dt=7), dict(act=2), dict(act=-1), dict(x=None), dict(wg=None), dict(wu=None), dict(wd=None), dict(out=None), dict(work=None),
               dict(nbytes=100), dict(work=(6 << 40) + 16), dict(d=(1 << 24) + 1), dict(f=1 << 25), dict(n=1 << 40), dict(saved=(7 << 40) + 2)):
        assert _ffn(L, **kw) == INVALID, kw
    assert _ffn(L, dt=0) == UNSUPPORTED
    assert _ffn(L, out=1 << 40) == OVERLAP
    assert _ffn(L, saved=6 << 40) == OVERLAP
    assert _ffn(L, n=0) == 0
    for kw in (dict(dt=7), dict(act=2), dict(x=None), dict(dy=None), dict(saved=None), dict(wd=None), dict(work=None), dict(nbytes=100)):
        assert _ffn_grad(L, **kw) == INVALID, kw
    assert _ffn_grad(L, dt=0) == UNSUPPORTED
    assert _ffn_grad(L, dx=8 << 40) == OVERLAP
    assert _ffn_grad(L, dwu=10 << 40) == OVERLAP
    assert _ffn_grad(L, dx=None, dwg=None, dwu=None, dwd=None) == 0
    for kw in (dict(dt=3), dict(ls=99), dict(logits=None), dict(ids=None), dict(t=None), dict(loss=None), dict(top=1025), dict(tau=0.0), dict(tau=-1.0),
               dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e-39), dict(n=1 << 30), dict(v=1 << 31, ls=1 << 31), dict(grad=9 << 40, gs=99)):
        assert _distill(L, **kw) == INVALID, kw
    assert _distill(L, grad=(1 << 40) + 400) == OVERLAP      # shifted by a row
    assert _distill(L, grad=1 << 40, gs=104) == OVERLAP      # in place with another stride
    assert _distill(L, loss=(2 << 40)) == OVERLAP
    assert _distill(L, stats=(1 << 40)) == OVERLAP
    assert _distill(L, n=0) == 0
    for kw in (dict(dt=3), dict(stats=None), dict(grad=None), dict(gs=99), dict(top=2000)):
        assert _distill_grad(L, **kw) == INVALID, kw
    assert _distill_grad(L, grad=4 << 40) == OVERLAP
    z = ctypes.c_size_t()
    assert L.ccl_plan_gated_ffn_work_bytes(1, 1 << 25, 8, 0, 1, ctypes.byref(z)) == INVALID
    assert L.ccl_plan_gated_ffn_work_bytes(1, 8, 8, 0, 1, None) == INVALID
    assert L.ccl_plan_embedding_grad_work_bytes(1 << 31, 8, 8, ctypes.byref(z)) == INVALID
    assert L.ccl_plan_embedding_grad_work_bytes(8, 8, 8, None) == INVALID
    assert L.ccl_gated_ffn_timeouts(None) == INVALID


def test_c_entries_refuse_before_launching():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    res = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "refusals ok" in res.stdout


def test_plans():
    # two lists of (row, position) pairs, and two fp32 partial rows for every piece of 8 (few tokens) to 32 once there are two
    assert ccl.ccl_plan_embedding_grad_work_bytes(8, 1000, 4096) == 2 * 256
    assert ccl.ccl_plan_embedding_grad_work_bytes(64, 1000, 4096) == 2 * 512 + 2 * 8 * 4096 * 4
    assert ccl.ccl_plan_embedding_grad_work_bytes(1 << 20, 1000, 4096) == 2 * (8 << 20) + 2 * (1 << 15) * 4096 * 4
    # h alone; h, dg and du; padded copies where a width is no multiple of 8 or a base is unaligned
    t, d, f = 4096, 4096, 11008
    assert ccl.ccl_plan_gated_ffn_work_bytes(t, d, f) == t * f * 2
    assert ccl.ccl_plan_gated_ffn_work_bytes(t, d, f, backward=True) == 3 * t * f * 2
    weights = 3 * d * f * 2
    assert ccl.ccl_plan_gated_ffn_work_bytes(t, d, f, aligned=False) == t * f * 2 + weights + t * d * 2
    assert ccl.ccl_plan_gated_ffn_work_bytes(t, d, f, backward=True, aligned=False) == 3 * t * f * 2 + weights + 2 * t * d * 2
    assert ccl.ccl_plan_gated_ffn_work_bytes(t, d - 1, f) == t * f * 2 + 2 * d * f * 2 + t * d * 2
    for t, d, f in ((1, 4096, 11008), (48, 300, 700), (300, 1001, 2733), (5000, 64, 64), (2000, 512, 1376), (200, 8, 20000)):
        # a backward pass's buffer serves the forward too
        assert ccl.ccl_plan_gated_ffn_work_bytes(t, d, f, backward=True) >= ccl.ccl_plan_gated_ffn_work_bytes(t, d, f)


def test_binding_names_what_is_wrong():
    cpu = torch.zeros(4, 8)
    ids = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        ccl.ccl_embedding(cpu, ids, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ccl.ccl_distill_loss(cpu, ids.view(4, 1), torch.zeros(4, 1), torch.zeros(4))
    with pytest.raises(ValueError, match="contiguous rows"):
        C._rows(cpu.t(), "table")
    with pytest.raises(ValueError, match="columns"):
        C._rows(cpu, "out", 7)
    with pytest.raises(TypeError, match="int64"):
        C._flat(ids.int(), "ids", (4,), torch.int64)
    with pytest.raises(ValueError, match="shape"):
        C._flat(ids, "ids", (5,), torch.int64)
    assert C._rows(torch.zeros(3, 10)[:, :4], "t")[1:] == (3, 4, 10)
    assert C._rows(torch.zeros(1, 10)[:, :4], "t")[1:] == (1, 4, 4)
    with pytest.raises(KeyError):
        C._act("relu")


if __name__ == "__main__":
    refusals(ccl.lib())
    print("refusals ok")
