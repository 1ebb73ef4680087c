"""The feed-forward block where a CTA, or a pair of them, takes several tiles:
both accumulators in turn, their release, and the ring of stages going on from
one tile to the next, in every kernel and epilogue.  (The other tests' shapes
give most of them one tile.)  Same bounds as there."""
import importlib.util
import os

import pytest

_spec = importlib.util.spec_from_file_location("gated_ffn_bounds", os.path.join(os.path.dirname(os.path.abspath(__file__)), "test_gpu_gated_ffn.py"))
base = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(base)

pytestmark = pytest.mark.gpu

# few tokens on 152 CTAs: g and u in 625 tiles (5 a CTA) and dh in 313 (3), then y and dx in 313; odd rows; and the layer of
# one token, whose g and u are cut into 7 parts along K (602 of them, 4 a CTA), and of a decode batch
FEW = [(5, 72, 80000), (5, 80000, 72), (30, 129, 40001), (30, 40001, 129), (1, 4096, 11008), (48, 4096, 11008)]
# many tokens on 76 pairs: g and u in 360 tiles (5 a pair) and dh in 180 (3), then y and dx in 180, rows of vectors and odd
# rows; the weights' gradients in 240; all of these whole, not cut along K
MANY = [(2100, 72, 5000), (2100, 5000, 72), (2100, 75, 5001), (2100, 5001, 75), (300, 2500, 1900)]


@pytest.mark.parametrize("T,D,F", FEW + MANY)
def test_several_tiles_for_each(T, D, F):
    args = base.inputs(T, D, F, T + D)
    base.check(base.forward_backward(*args, "silu"), base.reference(*args, "silu"))
