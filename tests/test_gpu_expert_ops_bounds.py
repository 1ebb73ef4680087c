"""The expert-parallel operators' tests again against the bounds-checking debug
build: every global load and store of their kernels stays inside the call's own
buffers (the tensor-memory copies of the feed-forward blocks, which the checks
do not see, are bounded by their tensor maps)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RUNNER = os.path.join(ROOT, "tests", "debug_bounds_run.py")

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

FILES = ["tests/test_gpu_route.py", "tests/test_gpu_dispatch.py", "tests/test_gpu_act8.py", "tests/test_gpu_expert_ffn.py"]


def test_every_access_stays_inside_the_calls_buffers():
    from ring_allreduce_rank_gb300 import build
    env = dict(os.environ, CCL_LIBRARY=build.build(debug_bounds=True))
    # not the graph tests: the range table is uploaded with a copy per call
    res = subprocess.run([sys.executable, RUNNER, "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", "-k", "not graph", *FILES], cwd=ROOT,
                         env=env, capture_output=True, text=True, timeout=3000)
    line = [l for l in res.stdout.splitlines() if l.startswith("DEBUG_FAULTS")]
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-2000:]
    assert line and int(line[-1].split()[1]) == 0, res.stdout[-2000:]
