"""The expert-parallel operators' argument checks, without a GPU: the C entries
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
NAN = float("nan")
T40 = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    from ring_allreduce_rank_gb300 import build
    build.build()
    ccl.lib()


def _route(L, z=1 * T40, n=1000, e=8, zs=8, dt=0, valid=None, top=2, norm=1, ids=2 * T40, w=3 * T40, lse=4 * T40, counts=5 * T40, load=6 * T40,
           imp=7 * T40, loss=8 * T40, work=9 * T40, nbytes=1 << 20):
    return L.ccl_route(z, n, e, zs, dt, valid, top, norm, ids, w, lse, counts, load, imp, loss, work, nbytes, None)


def _route_grad(L, z=1 * T40, n=100, e=8, zs=8, dt=0, ids=2 * T40, top=2, norm=1, lse=4 * T40, counts=5 * T40, load=6 * T40, gw=3 * T40, b=0.0, c=0.0,
                grad=9 * T40, gs=8):
    return L.ccl_route_grad(z, n, e, zs, dt, ids, top, norm, lse, counts, load, gw, b, c, grad, gs, None)


def _order(L, ids=1 * T40, n=50000, top=2, first=0, e=8, off=2 * T40, place=3 * T40, work=4 * T40, nbytes=1 << 24):
    return L.ccl_expert_order(ids, n, top, first, e, off, place, work, nbytes, None)


def _dispatch(L, x=1 * T40, n=10, dim=8, xs=8, dt=0, place=2 * T40, top=2, rows=3 * T40, nrows=20, rs=8):
    return L.ccl_dispatch(x, n, dim, xs, dt, place, top, rows, nrows, rs, None)


def _combine(L, rows=3 * T40, nrows=20, dim=8, rs=8, dt=0, place=2 * T40, w=4 * T40, n=10, top=2, out=1 * T40, os_=8):
    return L.ccl_combine(rows, nrows, dim, rs, dt, place, w, n, top, out, os_, None)


def _combine_grad(L, dy=1 * T40, ys=8, rows=3 * T40, nrows=20, dim=8, rs=8, dt=0, place=2 * T40, w=4 * T40, n=10, top=2, gr=5 * T40, gs=8, gw=6 * T40):
    return L.ccl_combine_grad(dy, ys, rows, nrows, dim, rs, dt, place, w, n, top, gr, gs, gw, None)


def _pack(L, x=1 * T40, n=4, c=40, xs=40, dt=0, codes=2 * T40, scales=3 * T40):
    return L.ccl_act8_pack(x, n, c, xs, dt, codes, scales, None)


def _unpack(L, x=1 * T40, n=4, c=40, xs=40, dt=0, codes=2 * T40, scales=3 * T40):
    return L.ccl_act8_unpack(codes, scales, n, c, dt, x, xs, None)


def _ffn(L, x=1 * T40, off=7 * T40, wg=2 * T40, wu=3 * T40, wd=4 * T40, n=4, e=2, d=16, f=24, dt=1, act=0, out=5 * T40, codes=None, scales=None, work=6 * T40,
         nbytes=1 << 26):
    return L.ccl_expert_ffn(x, off, wg, wu, wd, n, e, d, f, dt, act, out, codes, scales, work, nbytes, None)


def _ffn_grad(L, dy=1 * T40, x=2 * T40, xc=None, xsc=None, off=3 * T40, wg=4 * T40, wu=5 * T40, wd=6 * T40, codes=7 * T40, scales=8 * T40, n=4, e=2, d=16, f=24,
              dt=1, act=0, acc=0, dx=9 * T40, dwg=10 * T40, dwu=11 * T40, dwd=12 * T40, work=13 * T40, nbytes=1 << 26):
    return L.ccl_expert_ffn_grad(dy, x, xc, xsc, off, wg, wu, wd, codes, scales, n, e, d, f, dt, act, acc, dx, dwg, dwu, dwd, work, nbytes, None)


def refusals(L):
    for kw in (dict(dt=2), dict(zs=7), dict(e=0, zs=0), dict(e=1025, zs=1025), dict(top=0), dict(top=9), dict(e=64, zs=64, top=33), dict(n=1 << 31), dict(z=None),
               dict(ids=None), dict(w=None), dict(lse=None), dict(counts=None), dict(load=None), dict(imp=None), dict(loss=None), dict(work=None), dict(nbytes=0),
               dict(work=9 * T40 + 16), dict(z=T40 + 2), dict(ids=2 * T40 + 2), dict(zs=1 << 62), dict(n=1 << 30, nbytes=1 << 40)):
        assert _route(L, **kw) == INVALID, kw
    for kw in (dict(ids=T40 + 8), dict(load=6 * T40 + 4, imp=6 * T40), dict(lse=3 * T40), dict(valid=4 * T40), dict(work=5 * T40)):
        assert _route(L, **kw) == OVERLAP, kw
    for kw in (dict(dt=2), dict(zs=7), dict(gs=7), dict(top=0), dict(top=9), dict(b=NAN), dict(c=NAN), dict(z=None), dict(ids=None), dict(lse=None), dict(counts=None),
               dict(load=None), dict(gw=None), dict(grad=None), dict(grad=9 * T40 + 1), dict(e=2000, zs=2000, gs=2000), dict(n=1 << 30)):
        assert _route_grad(L, **kw) == INVALID, kw
    for kw in (dict(grad=T40 + 32), dict(grad=T40, gs=9), dict(grad=2 * T40), dict(grad=6 * T40)):
        assert _route_grad(L, **kw) == OVERLAP, kw
    assert _route_grad(L, n=0) == 0
    for kw in (dict(ids=None), dict(off=None), dict(place=None), dict(work=None), dict(nbytes=8), dict(work=4 * T40 + 8), dict(top=33), dict(e=1025), dict(n=1 << 31),
               dict(n=1 << 27, top=16), dict(off=2 * T40 + 2)):
        assert _order(L, **kw) == INVALID, kw
    for kw in (dict(place=T40), dict(off=3 * T40), dict(work=3 * T40)):
        assert _order(L, **kw) == OVERLAP, kw
    for kw in (dict(dt=5), dict(xs=7), dict(rs=7), dict(x=None), dict(rows=None), dict(place=None), dict(top=33), dict(dim=(1 << 24) + 1, xs=1 << 25, rs=1 << 25),
               dict(nrows=1 << 31), dict(x=T40 + 2), dict(place=2 * T40 + 1), dict(rs=1 << 62)):
        assert _dispatch(L, **kw) == INVALID, kw
    assert _dispatch(L, rows=T40 + 64) == OVERLAP
    assert _dispatch(L, rows=2 * T40) == OVERLAP
    assert _dispatch(L, n=0) == 0 and _dispatch(L, nrows=0) == 0 and _dispatch(L, dim=0) == 0 and _dispatch(L, top=0, place=None) == 0
    for kw in (dict(dt=5), dict(rs=7), dict(os_=7), dict(rows=None), dict(out=None), dict(place=None), dict(w=4 * T40 + 2), dict(top=33), dict(n=1 << 31)):
        assert _combine(L, **kw) == INVALID, kw
    assert _combine(L, out=3 * T40 + 64) == OVERLAP
    assert _combine(L, out=4 * T40) == OVERLAP
    assert _combine(L, n=0) == 0
    for kw in (dict(dt=5), dict(ys=7), dict(rs=7), dict(gs=7), dict(dy=None), dict(rows=None), dict(place=None), dict(top=33), dict(gr=5 * T40 + 2), dict(gw=6 * T40 + 2)):
        assert _combine_grad(L, **kw) == INVALID, kw
    for kw in (dict(gr=3 * T40 + 32), dict(gr=3 * T40, gs=9), dict(gr=T40), dict(gw=4 * T40), dict(gw=5 * T40)):
        assert _combine_grad(L, **kw) == OVERLAP, kw
    assert _combine_grad(L, gr=None, gw=None) == 0
    for fn in (_pack, _unpack):
        for kw in (dict(dt=4), dict(xs=39), dict(x=None), dict(codes=None), dict(scales=None), dict(codes=2 * T40 + 16), dict(x=T40 + 2), dict(n=1 << 31),
                   dict(c=(1 << 24) + 1, xs=1 << 25)):
            assert fn(L, **kw) == INVALID, kw
        assert fn(L, codes=T40) == OVERLAP
        assert fn(L, n=0) == 0 and fn(L, c=0) == 0
    assert _pack(L, scales=2 * T40 + 64) == OVERLAP
    for kw in (dict(dt=7), dict(act=2), dict(act=-1), dict(x=None), dict(off=None), dict(wg=None), dict(wu=None), dict(wd=None), dict(out=None), dict(work=None),
               dict(nbytes=100), dict(work=6 * T40 + 16), dict(d=(1 << 24) + 1), dict(f=1 << 25), dict(f=0), dict(e=1025), dict(n=1 << 31), dict(codes=8 * T40),
               dict(scales=8 * T40), dict(codes=8 * T40 + 16, scales=9 * T40), dict(off=7 * T40 + 2), dict(x=T40 + 1)):
        assert _ffn(L, **kw) == INVALID, kw
    assert _ffn(L, dt=0) == UNSUPPORTED
    for kw in (dict(out=1 * T40), dict(out=7 * T40), dict(codes=6 * T40, scales=8 * T40), dict(codes=8 * T40, scales=8 * T40 + 32)):
        assert _ffn(L, **kw) == OVERLAP, kw
    assert _ffn(L, n=0) == 0 and _ffn(L, e=0) == 0 and _ffn(L, d=0) == 0
    for kw in (dict(dt=7), dict(act=2), dict(x=None), dict(x=None, xc=14 * T40), dict(x=None, xc=14 * T40 + 8, xsc=15 * T40), dict(dy=None), dict(off=None),
               dict(codes=None), dict(scales=None), dict(wd=None), dict(work=None), dict(nbytes=100), dict(f=0)):
        assert _ffn_grad(L, **kw) == INVALID, kw
    assert _ffn_grad(L, dt=0) == UNSUPPORTED
    for kw in (dict(dx=T40), dict(dwu=10 * T40), dict(x=None, xc=9 * T40, xsc=15 * T40), dict(dwd=7 * T40)):
        assert _ffn_grad(L, **kw) == OVERLAP, kw
    assert _ffn_grad(L, dx=None, dwg=None, dwu=None, dwd=None) == 0
    z = ctypes.c_size_t()
    assert L.ccl_plan_route_work_bytes(1, 1025, ctypes.byref(z)) == INVALID
    assert L.ccl_plan_route_work_bytes(1, 8, None) == INVALID
    assert L.ccl_plan_expert_order_work_bytes(1, 33, 8, ctypes.byref(z)) == INVALID
    assert L.ccl_plan_expert_order_work_bytes(1, 3, 8, None) == INVALID
    assert L.ccl_plan_act8_width((1 << 24) + 1, ctypes.byref(z)) == INVALID
    assert L.ccl_plan_act8_width(8, None) == INVALID
    assert L.ccl_plan_expert_ffn_work_bytes(8, 8, 8, 1 << 25, 0, 1, ctypes.byref(z)) == INVALID
    assert L.ccl_plan_expert_ffn_work_bytes(8, 8, 8, 8, 0, 1, None) == INVALID


def test_c_entries_refuse_before_launching():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    res = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "refusals ok" in res.stdout


def test_plans():
    assert [ccl.ccl_plan_act8_width(c) for c in (0, 1, 32, 33, 11008)] == [0, 32, 32, 64, 11008]
    # one CTA needs no working space; several leave a row of sums each
    assert ccl.ccl_plan_route_work_bytes(8, 256) == 0 and ccl.ccl_plan_route_work_bytes(128, 64) == 0
    assert ccl.ccl_plan_route_work_bytes(1 << 20, 256) == -(-152 * 257 * 4 // 256) * 256 + -(-152 * 258 * 4 // 256) * 256
    assert ccl.ccl_plan_expert_order_work_bytes(2048, 8, 64) == 0
    assert ccl.ccl_plan_expert_order_work_bytes(65537, 1, 64) == 64 * 1025 * 4 + 256  # 1025 runs of 64
    # backward: h, dg and du in rows of whole blocks, and x and grad_out, every expert's rows padded to a multiple of 64
    r, e, d, f = 1000, 4, 512, 776
    padded = -(-(r + 63 * e) // 64) * 64
    assert ccl.ccl_plan_expert_ffn_work_bytes(r, e, d, f, backward=True) == padded * (3 * 800 + 2 * 512) * 2
    assert ccl.ccl_plan_expert_ffn_work_bytes(r, e, d, f) == r * 800 * 2
    for args in ((1, 8, 4096, 11008), (300, 5, 1001, 733), (64, 64, 2048, 1408), (50, 1, 64, 64), (5000, 1, 64, 64), (20, 1024, 8, 8)):
        # a backward pass's buffer serves the forward too
        assert ccl.ccl_plan_expert_ffn_work_bytes(*args, backward=True) >= ccl.ccl_plan_expert_ffn_work_bytes(*args)


def test_binding_names_what_is_wrong():
    f, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ccl.ccl_dispatch(f, i, f)
    with pytest.raises(TypeError, match="int32"):
        C._choices(i.long(), "ids")
    with pytest.raises(ValueError, match="top"):
        C._choices(i[0], "ids")
    with pytest.raises(ValueError, match="codes"):
        C._act8((torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8)), "x", (4,), 33)
    with pytest.raises(TypeError, match="scales"):
        C._act8((torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2)), "x", (4,), 33)
    w = torch.zeros(3, 6, 8)
    with pytest.raises(ValueError, match="w_down"):
        C._expert_shapes(f, torch.zeros(4, dtype=torch.int32), w, w, w)
    with pytest.raises(ValueError, match="offsets"):
        C._expert_shapes(f, torch.zeros(3, dtype=torch.int32), w, w, torch.zeros(3, 8, 6))


if __name__ == "__main__":
    refusals(ccl.lib())
    print("refusals ok")
