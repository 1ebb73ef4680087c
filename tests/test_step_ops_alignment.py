"""The training-step operators' C entries refuse pointers that are no multiple
of their element's size: the kernels' element loads would fault on them.  In a
child process that sees no GPU, on fake pointers that are never dereferenced."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, FP32, BF16 = 1, 0, 1
N, D, F, V, K = 4, 16, 24, 100, 5


def _embedding(L, dt, p):
    return L.ccl_embedding(p["table"], V, D, D, dt, p["ids"], N, 0, 1.0, p["out"], D, None)


def _embedding_grad(L, dt, p):
    return L.ccl_embedding_grad(p["dy"], D, p["ids"], N, 0, V, D, dt, 1.0, 0, p["grad"], D, p["work"], 1 << 20, None)


def _ffn(L, dt, p):
    return L.ccl_gated_ffn(p["x"], p["wg"], p["wu"], p["wd"], N, D, F, dt, 0, p["out"], p["saved"], p["work"], 1 << 26, None)


def _ffn_grad(L, dt, p):
    return L.ccl_gated_ffn_grad(p["dy"], p["x"], p["wg"], p["wu"], p["wd"], p["saved"], N, D, F, dt, 0, 0, p["dx"], p["dwg"], p["dwu"],
                                p["dwd"], p["work"], 1 << 26, None)


def _distill(L, dt, p):
    return L.ccl_distill_loss(p["logits"], N, V, V, dt, p["ids"], p["teacher"], K, 1.0, p["weights"], p["loss"], p["stats"], p["grad"], V,
                              None)


def _distill_grad(L, dt, p):
    return L.ccl_distill_grad(p["logits"], N, V, V, dt, p["ids"], p["teacher"], K, 1.0, p["weights"], p["stats"], p["grad"], V, None)


# the entry, its types, and each pointer's element size (0: the values' own)
ENTRIES = [
    (_embedding, (FP32, BF16), dict(table=0, ids=8, out=0)),
    (_embedding_grad, (FP32, BF16), dict(dy=0, ids=8, grad=0, work=16)),
    (_ffn, (BF16,), dict(x=0, wg=0, wu=0, wd=0, out=0, saved=4, work=256)),
    (_ffn_grad, (BF16,), dict(dy=0, x=0, wg=0, wu=0, wd=0, saved=4, dx=0, dwg=0, dwu=0, dwd=0, work=256)),
    (_distill, (FP32, BF16), dict(logits=0, ids=8, teacher=4, weights=4, loss=4, stats=4, grad=0)),
    (_distill_grad, (FP32, BF16), dict(logits=0, ids=8, teacher=4, weights=4, stats=4, grad=0)),
]


def refusals(L):
    for entry, types, sizes in ENTRIES:
        for dt in types:
            sound = {k: (i + 1) << 40 for i, k in enumerate(sizes)}
            # without a GPU a sound call gets past the checks and fails at its launch
            assert entry(L, dt, sound) != INVALID, entry.__name__
            for name, size in sizes.items():
                size = size or (4 if dt == FP32 else 2)
                for off in {1, size // 2}:
                    assert entry(L, dt, {**sound, name: sound[name] + off}) == INVALID, (entry.__name__, dt, name, off)


def test_pointers_off_their_elements_boundary_are_refused():
    from ring_allreduce_rank_gb300 import build
    build.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    res = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "refusals ok" in res.stdout


if __name__ == "__main__":
    import ring_allreduce_rank_gb300 as ccl
    refusals(ccl.lib())
    print("refusals ok")
