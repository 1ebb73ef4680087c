"""Cases of the training-step operators: embedding, gated feed-forward block, distillation loss.

Each case is one call (or one forward and backward pair) that a data-parallel rank makes to produce the gradients it
then reduces.  ``own`` picks between the library's kernels and the same operators in elementary torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, FP32 = torch.bfloat16, torch.float32
# the layer of the bucketed-gradient workload: hidden and feed-forward widths
HIDDEN, FFN = 4096, 11008


def listed():
    return [
        # one decoding step's token ids of a small batch: launch latency
        {"name": "embed_decode", "op": "embed", "dtype": "bf16", "tokens": 8, "rows": 32000, "dim": HIDDEN},
        # a long prompt batch: every row a gather of 8 KiB
        {"name": "embed_prompt", "op": "embed", "dtype": "bf16", "tokens": 16384, "rows": 32000, "dim": HIDDEN},
        # a short sequence's gradient in fp32 with a width that no vector load divides
        {"name": "embed_grad_short", "op": "embed_grad", "dtype": "fp32", "tokens": 500, "rows": 8011, "dim": 1031},
        # a training batch: Zipf-distributed ids, so a few rows take many tokens and most take none
        {"name": "embed_grad_batch", "op": "embed_grad", "dtype": "bf16", "tokens": 16384, "rows": 32000, "dim": HIDDEN},
        # one token of one request: the weights are read once for it
        {"name": "ffn_token", "op": "ffn", "tokens": 1, "dim": HIDDEN, "ffn": FFN, "act": "silu"},
        # one decoding step of a batch of requests
        {"name": "ffn_decode_batch", "op": "ffn", "tokens": 48, "dim": HIDDEN, "ffn": FFN, "act": "silu"},
        # a prompt batch: the matrix rate
        {"name": "ffn_prompt", "op": "ffn", "tokens": 4096, "dim": HIDDEN, "ffn": FFN, "act": "silu"},
        # a rank's micro-batch, forward and backward
        {"name": "ffn_train", "op": "ffn_train", "tokens": 2048, "dim": HIDDEN, "ffn": FFN, "act": "silu"},
        # a small model with widths that no 16-byte row stride divides
        {"name": "ffn_train_odd", "op": "ffn_train", "tokens": 301, "dim": 1001, "ffn": 2733, "act": "gelu"},
        # the loss alone, of a few positions (a validation probe): launch latency
        {"name": "distill_short", "op": "distill", "dtype": "bf16", "tokens": 16, "vocab": 32000, "top": 32, "form": "loss", "tau": 1.0},
        # a training batch over a large vocabulary, loss and gradient in one call
        {"name": "distill_train", "op": "distill", "dtype": "bf16", "tokens": 4096, "vocab": 128000, "top": 64, "form": "fused", "tau": 2.0},
        # forward first, backward when its turn comes, fp32 logits with an odd row length
        {"name": "distill_odd", "op": "distill", "dtype": "fp32", "tokens": 333, "vocab": 50257, "top": 20, "form": "two", "tau": 1.5},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step, its logarithm uniform; the round multiples of 1024 are the listed cases' ground."""
    v = max(step, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) // step * step)
    return v - step if v % 1024 == 0 else v


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "ffn", "ffn_train", "distill", "distill"])
    if op in ("embed", "embed_grad"):
        dim = _log(rng, 64, HIDDEN, 1 if rng.random() < 0.3 else 8)
        dtype = rng.choice(["bf16", "fp32"])
        # fp32 rows weigh twice as much: half the rows and tokens keep a case within the listed ones
        most = 1 if dtype == "bf16" else 2
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 16384 // most), "rows": _log(rng, 500, 32000 // most), "dim": dim}
    if op in ("ffn", "ffn_train"):
        step = 1 if rng.random() < 0.3 else 8
        dim, ffn = _log(rng, 200, HIDDEN, step), _log(rng, 500, FFN, step)
        return {"op": op, "tokens": _log(rng, 1, 4096 if op == "ffn" else 2048), "dim": dim, "ffn": ffn, "act": rng.choice(["silu", "gelu"])}
    vocab = _log(rng, 1000, 128000, 1 if rng.random() < 0.5 else 8)
    dtype = rng.choice(["bf16", "fp32"])
    return {"op": "distill", "dtype": dtype, "tokens": _log(rng, 1, 4096 if dtype == "bf16" else 2048), "vocab": vocab,
            "top": min(_log(rng, 1, 256), vocab), "form": rng.choice(["loss", "fused", "two"]), "tau": rng.choice([1.0, 1.5, 2.0, 4.0])}


def _dt(name):
    return {"bf16": BF16, "fp32": FP32}[name]


def _randn(gen, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=gen, device=DEV, dtype=FP32) * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    s = dict(case)
    op = case["op"]
    if op in ("embed", "embed_grad"):
        T, V, D, dt = case["tokens"], case["rows"], case["dim"], _dt(case["dtype"])
        # log-uniform ranks over a shuffled vocabulary (Zipf with exponent 1); a padding id now and then
        u = torch.rand(T, generator=gen, device=DEV, dtype=torch.float64)
        rank = (torch.exp(u * math.log(V)) - 1).long().clamp_(0, V - 1)
        ids = torch.randperm(V, generator=gen, device=DEV)[rank]
        ids[torch.rand(T, generator=gen, device=DEV) < 0.02] = -1
        s["ids"], s["scale"] = ids.contiguous(), math.sqrt(D)
        if op == "embed":
            s["table"] = _randn(gen, V, D, std=0.02, dtype=dt)
            s["out"] = torch.empty(T, D, device=DEV, dtype=dt)
        else:
            s["grad_out"] = _randn(gen, T, D, std=1e-3, dtype=dt)
            s["grad_table"] = torch.empty(V, D, device=DEV, dtype=dt)
            if own:
                import ring_allreduce_rank_gb300 as ccl
                s["work"] = torch.empty(ccl.ccl_plan_embedding_grad_work_bytes(T, V, D), dtype=torch.uint8, device=DEV)
    elif op in ("ffn", "ffn_train"):
        T, D, F = case["tokens"], case["dim"], case["ffn"]
        s["x"] = _randn(gen, T, D)
        s["wg"], s["wu"] = _randn(gen, F, D, std=D ** -0.5), _randn(gen, F, D, std=D ** -0.5)
        s["wd"] = _randn(gen, D, F, std=F ** -0.5)
        s["out"] = torch.empty(T, D, device=DEV, dtype=BF16)
        if op == "ffn_train":
            s["dy"] = _randn(gen, T, D, std=1e-2)
            s["dx"] = torch.empty(T, D, device=DEV, dtype=BF16)
            s["dwg"], s["dwu"] = torch.empty(F, D, device=DEV, dtype=BF16), torch.empty(F, D, device=DEV, dtype=BF16)
            s["dwd"] = torch.empty(D, F, device=DEV, dtype=BF16)
        if own:
            import ring_allreduce_rank_gb300 as ccl
            nbytes = ccl.ccl_plan_gated_ffn_work_bytes(T, D, F, backward=op == "ffn_train")
            s["work"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
            s["saved"] = torch.empty(2, T, F, device=DEV, dtype=FP32) if op == "ffn_train" else None
    else:
        T, V, K, dt = case["tokens"], case["vocab"], case["top"], _dt(case["dtype"])
        logits = torch.randn(T, V, generator=gen, device=DEV, dtype=FP32) * 1.5
        ids = torch.randint(0, V, (T, K), generator=gen, device=DEV)
        # the teacher's own order; the student follows it with noise
        teacher = (torch.randn(T, K, generator=gen, device=DEV) * 2 + 8).sort(dim=1, descending=True).values
        student = teacher + torch.randn(T, K, generator=gen, device=DEV) * 1.5 - 1
        logits.scatter_reduce_(1, ids, student, "amax", include_self=False)  # an id may come twice
        logits[:, V - 3:] = float("-inf")  # vocabulary padding
        ids[ids >= V - 3] = 0
        row = torch.rand(T, generator=gen, device=DEV)
        # short lists (the rest marked -1, whatever their logits hold), and positions without a teacher
        short = torch.rand(T, K, generator=gen, device=DEV) < 0.1
        ids[short] = -1
        teacher[short] = float("nan")
        ids[row < 0.04] = -1
        weights = torch.full((T,), 1.0 / T, device=DEV)
        weights[row > 0.95] = 0.0  # positions left out of the loss
        s["logits"], s["ids"], s["teacher"], s["weights"] = logits.to(dt), ids, teacher.contiguous(), weights
        s["loss"], s["stats"] = torch.empty(T, device=DEV), torch.empty(T, 2, device=DEV)
        if case["form"] != "loss":
            s["grad"] = torch.empty(T, V, device=DEV, dtype=dt)
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import ring_allreduce_rank_gb300 as ccl
    op = s["op"]
    if op == "embed":
        ccl.ccl_embedding(s["table"], s["ids"], s["out"], scale=s["scale"])
        return s["out"]
    if op == "embed_grad":
        ccl.ccl_embedding_grad(s["grad_out"], s["ids"], s["grad_table"], scale=s["scale"], work=s["work"])
        return s["grad_table"]
    if op == "ffn":
        ccl.ccl_gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], s["out"], act=s["act"], work=s["work"])
        return s["out"]
    if op == "ffn_train":
        ccl.ccl_gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], s["out"], act=s["act"], saved=s["saved"], work=s["work"])
        ccl.ccl_gated_ffn_grad(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], s["saved"], s["dx"], s["dwg"], s["dwu"], s["dwd"],
                               act=s["act"], work=s["work"])
        return {k: s[k] for k in ("out", "dx", "dwg", "dwu", "dwd")}
    a = (s["logits"], s["ids"], s["teacher"])
    if s["form"] == "two":
        ccl.ccl_distill_loss(*a, s["loss"], stats=s["stats"], weights=s["weights"], temperature=s["tau"])
        ccl.ccl_distill_grad(*a, s["stats"], s["grad"], weights=s["weights"], temperature=s["tau"])
        return {"loss": s["loss"], "grad": s["grad"]}
    if s["form"] == "fused":
        ccl.ccl_distill_loss(*a, s["loss"], grad=s["grad"], weights=s["weights"], temperature=s["tau"])
        return {"loss": s["loss"], "grad": s["grad"]}
    ccl.ccl_distill_loss(*a, s["loss"], weights=s["weights"], temperature=s["tau"])
    return {"loss": s["loss"]}


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


def _run_plain(s):
    op = s["op"]
    if op == "embed":
        ids, table = s["ids"], s["table"]
        ok = (ids >= 0) & (ids < table.shape[0])
        rows = table[torch.where(ok, ids, 0)].float() * s["scale"]
        return (rows * ok[:, None]).to(table.dtype)
    if op == "embed_grad":
        ids, dy = s["ids"], s["grad_out"]
        V = s["rows"]
        ok = (ids >= 0) & (ids < V)
        acc = torch.zeros(V, dy.shape[1], device=dy.device, dtype=FP32)
        acc.index_add_(0, torch.where(ok, ids, 0), dy.float() * ok[:, None])
        return (acc * s["scale"]).to(dy.dtype)
    if op in ("ffn", "ffn_train"):
        x, wg, wu, wd = (s[k].float() for k in ("x", "wg", "wu", "wd"))
        g, u = x @ wg.t(), x @ wu.t()
        a, da = _act(g, s["act"])
        h = a * u
        y = (h @ wd.t()).to(BF16)
        if op == "ffn":
            return y
        dy = s["dy"].float()
        dh = dy @ wd
        dg, du = dh * u * da, dh * a
        grads = {"dx": dg @ wg + du @ wu, "dwg": dg.t() @ x, "dwu": du.t() @ x, "dwd": dy.t() @ h}
        return {"out": y, **{k: v.to(BF16) for k, v in grads.items()}}
    z = s["logits"].float() / s["tau"]
    ids, w = s["ids"], s["weights"]
    ok = (ids >= 0) & (ids < z.shape[1])
    at = torch.where(ok, ids, 0)
    t = torch.where(ok, s["teacher"] / s["tau"], -math.inf)
    tm = t.max(dim=1, keepdim=True).values
    some = tm > -math.inf
    e = torch.where(ok, torch.exp(t - torch.where(some, tm, 0.0)), 0.0)
    total = torch.where(some, e.sum(dim=1, keepdim=True), 1.0)
    p = e / total
    m = z.max(dim=1, keepdim=True).values
    ez = torch.exp(z - m)
    sum_z = ez.sum(dim=1, keepdim=True)
    term = p * ((t - tm) - torch.log(total) - (z.gather(1, at) - m) + torch.log(sum_z))
    loss = torch.where(p > 0, term, 0.0).sum(dim=1)
    loss = torch.where(w != 0, w * loss, 0.0)
    if s["form"] == "loss":
        return {"loss": loss}
    grad = ez / sum_z * some
    grad.scatter_add_(1, at, -p)
    grad = torch.where((w != 0)[:, None], grad * (w / s["tau"])[:, None], 0.0)
    return {"loss": loss, "grad": grad.to(s["logits"].dtype)}


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        T, V, D, e = case["tokens"], case["rows"], case["dim"], 2 if case["dtype"] == "bf16" else 4
        if op == "embed":
            return {"bytes": T * 8 + min(T, V) * D * e + T * D * e, "flops": T * D}
        return {"bytes": T * 8 + T * D * e + V * D * e, "flops": T * D}
    if op in ("ffn", "ffn_train"):
        T, D, F = case["tokens"], case["dim"], case["ffn"]
        if op == "ffn":
            return {"bytes": 2 * (3 * D * F + 2 * T * D), "flops": 6 * T * D * F}
        return {"bytes": 2 * (6 * D * F + 4 * T * D), "flops": 18 * T * D * F}
    T, V, K, e = case["tokens"], case["vocab"], case["top"], 2 if case["dtype"] == "bf16" else 4
    once = T * V * e + T * K * 12 + T * 8
    return {"bytes": once + (0 if case["form"] == "loss" else T * V * e), "flops": (4 if case["form"] == "loss" else 7) * T * V}


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "embed":
        padded = torch.cat([s["table"].to(f64), torch.zeros(1, case["dim"], device=DEV, dtype=f64)])
        ids = s["ids"].clone()
        ids[(ids < 0) | (ids >= case["rows"])] = case["rows"]
        return padded.index_select(0, ids) * s["scale"]
    if op == "embed_grad":
        ids = s["ids"].clone()
        ids[(ids < 0) | (ids >= case["rows"])] = case["rows"]
        acc = torch.zeros(case["rows"] + 1, case["dim"], device=DEV, dtype=f64)
        acc.index_put_((ids,), s["grad_out"].to(f64) * s["scale"], accumulate=True)
        return acc[:-1]
    if op in ("ffn", "ffn_train"):
        train = op == "ffn_train"
        x, wg, wu, wd = (s[k].to(f64).requires_grad_(train) for k in ("x", "wg", "wu", "wd"))
        g = torch.nn.functional.linear(x, wg)
        act = torch.nn.functional.silu(g) if case["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        y = torch.nn.functional.linear(act * torch.nn.functional.linear(x, wu), wd)
        if not train:
            return y
        dx, dwg, dwu, dwd = torch.autograd.grad(y, (x, wg, wu, wd), s["dy"].to(f64))
        return {"out": y.detach(), "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}
    # by rows: the definition through log_softmax, one slice of positions at a time
    T, V, tau = case["tokens"], case["vocab"], case["tau"]
    loss = torch.zeros(T, device=DEV, dtype=f64)
    grad = None if case["form"] == "loss" else torch.zeros(T, V, device=DEV, dtype=f64)
    for a in range(0, T, 256):
        rows = slice(a, min(T, a + 256))
        logq = torch.log_softmax(s["logits"][rows].to(f64) / tau, dim=1)
        ids, w = s["ids"][rows], s["weights"][rows].to(f64)
        valid = (ids >= 0) & (ids < V)
        t = s["teacher"][rows].to(f64).masked_fill(~valid, -math.inf) / tau
        logp = torch.log_softmax(t, dim=1).masked_fill(~valid, -math.inf)
        p = logp.exp()
        has = valid.any(dim=1)
        safe = ids.clamp(0, V - 1)
        kl = (p * (logp - logq.gather(1, safe))).masked_fill(p == 0, 0.0).sum(dim=1)
        loss[rows] = kl.masked_fill(~has, 0.0) * w
        if grad is not None:
            d = logq.exp() * has[:, None].to(f64)
            d.scatter_add_(1, safe, -p)
            grad[rows] = d * (w / tau)[:, None]
    return {"loss": loss} if grad is None else {"loss": loss, "grad": grad}
