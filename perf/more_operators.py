"""Cases of the expert-parallel operators: router, dispatch and combine of tokens, the experts' feed-forward blocks, 8-bit activation checkpoints.

Each case is one call (or one run of calls) that a rank of an expert-parallel training or serving step makes around the
all-to-all exchange of its tokens.  ``own`` picks between the library's kernels and the same operators in elementary
torch operations.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, FP32, I32 = torch.bfloat16, torch.float32, torch.int32
# the dense layer's hidden and feed-forward widths, the exchanged tokens' width, and the exchange's number of experts
HIDDEN, FFN, WIDE, EXPERTS = 4096, 11008, 7168, 64
# an activation's block of 32 values shares one power of two
BLOCK = 32


def listed():
    return [
        # one decoding step of a small batch: launch latency
        {"name": "route_decode", "op": "route", "dtype": "bf16", "tokens": 8, "experts": EXPERTS, "top": 2, "normalize": True, "form": "loss"},
        # a training batch over many experts, with the balance and z losses' gradients; some rows are padding
        {"name": "route_train", "op": "route", "dtype": "fp32", "tokens": 16384, "experts": 256, "top": 8, "normalize": True, "form": "train"},
        # a decoding step's tokens put in expert order
        {"name": "dispatch_decode", "op": "dispatch", "dtype": "bf16", "tokens": 16, "dim": HIDDEN, "experts": EXPERTS, "top": 2},
        # a training batch's send buffer of the all-to-all exchange: every token read once and written to its experts' rows
        {"name": "dispatch_train", "op": "dispatch", "dtype": "bf16", "tokens": 8192, "dim": WIDE, "experts": EXPERTS, "top": 4},
        # a few fp32 tokens of a width that no vector load divides, summed back
        {"name": "combine_odd", "op": "combine", "dtype": "fp32", "tokens": 333, "dim": 1031, "experts": 10, "top": 3, "form": "forward"},
        # a training batch's weighted sum with the gradients by the experts' rows and by the weights
        {"name": "combine_train", "op": "combine", "dtype": "bf16", "tokens": 8192, "dim": WIDE, "experts": EXPERTS, "top": 4, "form": "train"},
        # one token of one request: the chosen experts' weights are read for it
        {"name": "experts_token", "op": "experts", "tokens": 1, "dim": HIDDEN, "ffn": FFN, "experts": 8, "top": 2, "act": "silu", "form": "forward"},
        # a prompt batch over eight large experts: the matrix rate
        {"name": "experts_prompt", "op": "experts", "tokens": 4096, "dim": HIDDEN, "ffn": FFN, "experts": 8, "top": 2, "act": "silu", "form": "forward"},
        # a micro-batch over many small experts, forward and backward through 8-bit checkpoints of x, g and u
        {"name": "experts_train", "op": "experts", "tokens": 8192, "dim": 2048, "ffn": 1408, "experts": 32, "top": 4, "act": "silu", "form": "train"},
        # a small model with widths that no 16-byte row stride divides
        {"name": "experts_train_odd", "op": "experts", "tokens": 150, "dim": 1001, "ffn": 733, "experts": 5, "top": 2, "act": "gelu", "form": "train"},
        # a short sequence's activations of an odd width, to 8 bits and back
        {"name": "act8_odd", "op": "act8", "dtype": "fp32", "rows": 200, "cols": 1001},
        # a feed-forward layer's activations of a micro-batch
        {"name": "act8_train", "op": "act8", "dtype": "bf16", "rows": 8192, "cols": FFN},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step, its logarithm uniform; the round multiples of 1024 are the listed cases' ground."""
    v = max(step, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) // step * step)
    return v - step if v % 1024 == 0 else v


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "experts", "experts", "act8"])
    dtype = rng.choice(["bf16", "fp32"])
    most = 1 if dtype == "bf16" else 2  # fp32 weighs twice as much
    step = 1 if rng.random() < 0.3 else 8
    if op == "route":
        experts = _log(rng, 4, 512, 1 if rng.random() < 0.3 else 4)
        top = min(_log(rng, 1, 12), experts)
        return {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 16384 * 256 // max(experts, 256)), "experts": experts, "top": top,
                "normalize": rng.random() < 0.7, "form": rng.choice(["loss", "train"])}
    if op in ("dispatch", "combine"):
        top = _log(rng, 1, 8)
        case = {"op": op, "dtype": dtype, "tokens": _log(rng, 1, 8192 * 4 // max(top, 4) // most), "dim": _log(rng, 64, WIDE, step),
                "experts": max(top, _log(rng, 2, 256)), "top": top}
        if op == "combine":
            case["form"] = rng.choice(["forward", "train"])
        return case
    if op == "experts":
        dim, ffn = _log(rng, 100, HIDDEN, step), _log(rng, 200, FFN, step)
        experts = _log(rng, 1, min(128, 8 * HIDDEN * FFN // (dim * ffn)))
        top = min(_log(rng, 1, 8), experts)
        form = rng.choice(["forward", "train"])
        # the listed ones' products at most
        rows = min(32768, (8192 if form == "forward" else 2700) * HIDDEN * FFN // (dim * ffn))
        return {"op": op, "tokens": _log(rng, 1, max(1, rows // top)), "dim": dim, "ffn": ffn, "experts": experts, "top": top,
                "act": rng.choice(["silu", "gelu"]), "form": form}
    cols = _log(rng, 64, FFN, step)
    return {"op": op, "dtype": dtype, "rows": _log(rng, 1, 8192 // most), "cols": cols}


def _dt(name):
    return {"bf16": BF16, "fp32": FP32}[name]


def _randn(gen, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=gen, device=DEV, dtype=FP32) * std).to(dtype)


def _choose(gen, T, E, K):
    """Distinct experts of every token, some experts more popular than others."""
    liking = torch.randn(T, E, generator=gen, device=DEV) + 0.4 * torch.randn(E, generator=gen, device=DEV)
    return liking.sort(dim=1, descending=True).indices[:, :K].to(I32).contiguous()


def _plan(ids, experts):
    """(offsets, place): the rows of the tokens' copies in expert order, -1 where there is none."""
    flat = ids.flatten().long()
    ok = (flat >= 0) & (flat < experts)
    key = torch.where(ok, flat, experts)
    order = key.sort(stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    ends = (key[:, None] < torch.arange(1, experts + 1, device=key.device)).sum(dim=0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    return offsets.to(I32), torch.where(ok, place, -1).to(I32).view(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 6007 + 29)
    s = dict(case)
    op = case["op"]
    if own:
        import ring_allreduce_rank_gb300 as ccl
    if op == "route":
        T, E, K, dt = case["tokens"], case["experts"], case["top"], _dt(case["dtype"])
        s["logits"] = (torch.randn(T, E, generator=gen, device=DEV) * 1.5 + 0.5 * torch.randn(E, generator=gen, device=DEV)).to(dt)
        s["logits"][:, 0] = s["logits"][:, E - 1]  # a tie in every row
        s["valid"] = (torch.rand(T, generator=gen, device=DEV) > 0.03).to(torch.uint8)  # the others are padding
        if T > 4:
            s["logits"][T // 2] = float("-inf")  # a row whose mask leaves no expert
        s["ids"] = torch.empty(T, K, device=DEV, dtype=I32)
        s["weights"], s["lse"] = torch.empty(T, K, device=DEV), torch.empty(T, device=DEV)
        s["counts"] = torch.empty(E + 1, device=DEV, dtype=I32)
        s["load"], s["importance"], s["loss"] = torch.empty(E, device=DEV), torch.empty(E, device=DEV), torch.empty(2, device=DEV)
        if case["form"] == "train":
            s["grad_weights"] = torch.randn(T, K, generator=gen, device=DEV) / T
            s["grad_logits"] = torch.empty(T, E, device=DEV, dtype=dt)
        if own:
            s["work"] = torch.empty(ccl.ccl_plan_route_work_bytes(T, E), dtype=torch.uint8, device=DEV)
    elif op in ("dispatch", "combine"):
        T, D, E, K, dt = case["tokens"], case["dim"], case["experts"], case["top"], _dt(case["dtype"])
        ids = _choose(gen, T, E, K)
        ids[torch.rand(T, generator=gen, device=DEV) < 0.03] = -1  # padding tokens go nowhere
        if op == "dispatch":
            s["x"], s["ids"] = _randn(gen, T, D, dtype=dt), ids
            s["offsets"] = torch.empty(E + 1, device=DEV, dtype=I32)
            s["place"] = torch.empty(T, K, device=DEV, dtype=I32)
            s["rows"] = torch.zeros(T * K, D, device=DEV, dtype=dt)
            if own:
                s["work"] = torch.empty(ccl.ccl_plan_expert_order_work_bytes(T, K, E), dtype=torch.uint8, device=DEV)
        else:
            s["place"] = _plan(ids, E)[1].contiguous()
            s["rows"] = _randn(gen, T * K, D, dtype=dt)
            s["weights"] = torch.softmax(torch.randn(T, K, generator=gen, device=DEV), dim=1)
            s["out"] = torch.empty(T, D, device=DEV, dtype=dt)
            if case["form"] == "train":
                s["grad_out"] = _randn(gen, T, D, std=1e-2, dtype=dt)
                s["grad_rows"] = torch.zeros(T * K, D, device=DEV, dtype=dt)
                s["grad_weights"] = torch.empty(T, K, device=DEV)
    elif op == "experts":
        T, D, F, E, K = (case[k] for k in ("tokens", "dim", "ffn", "experts", "top"))
        ids = _choose(gen, T, E, K)
        R = T * K
        s["offsets"] = _plan(ids, E)[0].contiguous()
        s["x"] = _randn(gen, R, D)
        s["wg"], s["wu"] = _randn(gen, E, F, D, std=D ** -0.5), _randn(gen, E, F, D, std=D ** -0.5)
        s["wd"] = _randn(gen, E, D, F, std=F ** -0.5)
        s["out"] = torch.empty(R, D, device=DEV, dtype=BF16)
        if case["form"] == "train":
            s["dy"] = _randn(gen, R, D, std=1e-2)
            s["dx"] = torch.empty(R, D, device=DEV, dtype=BF16)
            s["dwg"], s["dwu"] = torch.empty(E, F, D, device=DEV, dtype=BF16), torch.empty(E, F, D, device=DEV, dtype=BF16)
            s["dwd"] = torch.empty(E, D, F, device=DEV, dtype=BF16)
        if own:
            nbytes = ccl.ccl_plan_expert_ffn_work_bytes(R, E, D, F, backward=case["form"] == "train")
            s["work"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
            if case["form"] == "train":
                wd, wf = ccl.ccl_plan_act8_width(D), ccl.ccl_plan_act8_width(F)
                s["x8"] = (torch.empty(R, wd, dtype=torch.int8, device=DEV), torch.empty(R, wd // BLOCK, dtype=torch.uint8, device=DEV))
                s["saved"] = (torch.empty(2, R, wf, dtype=torch.int8, device=DEV), torch.empty(2, R, wf // BLOCK, dtype=torch.uint8, device=DEV))
        else:
            # the experts that have rows, and the most rows of one
            n = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
            s["active"] = torch.tensor([e for e in range(E) if n[e]], device=DEV)
            s["most"] = max(n)
    else:
        R, C, dt = case["rows"], case["cols"], _dt(case["dtype"])
        x = torch.randn(R, C, generator=gen, device=DEV)
        x = x * torch.exp(torch.randn(R, 1, generator=gen, device=DEV))  # rows of different size, some outliers, a row of zeros
        x[torch.rand(R, C, generator=gen, device=DEV) < 1e-3] *= 30
        x[R // 2] = 0
        s["x"], s["back"] = x.to(dt), torch.empty(R, C, device=DEV, dtype=dt)
        if own:
            w = ccl.ccl_plan_act8_width(C)
            s["x8"] = (torch.empty(R, w, dtype=torch.int8, device=DEV), torch.empty(R, w // BLOCK, dtype=torch.uint8, device=DEV))
    return s


# the losses' coefficients in the training step
BALANCE, ZLOSS = 1e-2, 1e-3


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import ring_allreduce_rank_gb300 as ccl
    op = s["op"]
    if op == "route":
        ccl.ccl_route(s["logits"], s["ids"], s["weights"], s["lse"], s["counts"], s["load"], s["importance"], s["loss"],
                      normalize=s["normalize"], valid=s["valid"], work=s["work"])
        out = {k: s[k] for k in ("ids", "weights", "counts", "load", "importance", "loss")}
        if s["form"] == "train":
            ccl.ccl_route_grad(s["logits"], s["ids"], s["lse"], s["counts"], s["load"], s["grad_weights"], s["grad_logits"],
                               normalize=s["normalize"], balance=BALANCE, z=ZLOSS)
            out["grad_logits"] = s["grad_logits"]
        return out
    if op == "dispatch":
        ccl.ccl_expert_order(s["ids"], s["offsets"], s["place"], work=s["work"])
        ccl.ccl_dispatch(s["x"], s["place"], s["rows"])
        return {k: s[k] for k in ("offsets", "place", "rows")}
    if op == "combine":
        ccl.ccl_combine(s["rows"], s["place"], s["out"], weights=s["weights"])
        if s["form"] == "forward":
            return {"out": s["out"]}
        ccl.ccl_combine_grad(s["grad_out"], s["place"], rows=s["rows"], weights=s["weights"], grad_rows=s["grad_rows"], grad_weights=s["grad_weights"])
        return {k: s[k] for k in ("out", "grad_rows", "grad_weights")}
    if op == "experts":
        w = (s["wg"], s["wu"], s["wd"])
        if s["form"] == "forward":
            ccl.ccl_expert_ffn(s["x"], s["offsets"], *w, s["out"], act=s["act"], work=s["work"])
            return {"out": s["out"]}
        ccl.ccl_act8_pack(s["x"], *s["x8"])
        ccl.ccl_expert_ffn(s["x"], s["offsets"], *w, s["out"], act=s["act"], saved=s["saved"], work=s["work"])
        ccl.ccl_expert_ffn_grad(s["dy"], s["x8"], s["offsets"], *w, s["saved"], s["dx"], s["dwg"], s["dwu"], s["dwd"], act=s["act"], work=s["work"])
        return {k: s[k] for k in ("out", "dx", "dwg", "dwu", "dwd")}
    ccl.ccl_act8_pack(s["x"], *s["x8"])
    ccl.ccl_act8_unpack(*s["x8"], s["back"])
    return {"back": s["back"]}


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


def _eight_bits(x):
    """What x keeps of its values in 8 bits: in blocks of 32 along a row, the nearest multiples of 2^e, 2^e the least power of two with
    |x| <= 127 2^e in the block."""
    C = x.shape[-1]
    wide = torch.nn.functional.pad(x, (0, -C % BLOCK)).unflatten(-1, (-1, BLOCK))
    most = wide.abs().amax(dim=-1, keepdim=True)
    m, e = torch.frexp(most)  # most = m 2^e, 0.5 <= m < 1, and 127 = (127/128) 2^7
    step = torch.ldexp(torch.ones_like(most), e - 7 + (m > 127 / 128).int())
    step = torch.where(most > 0, step, 1.0)
    return (torch.round(wide / step) * step).flatten(-2)[..., :C]


def _run_plain(s):
    op = s["op"]
    if op == "route":
        z, E, K, T = s["logits"].float(), s["experts"], s["top"], s["tokens"]
        m = z.amax(dim=1, keepdim=True)
        live = (m[:, 0] > -math.inf) & (s["valid"] != 0)
        m = torch.where(live[:, None], m, 0.0)
        ez = torch.where(live[:, None], torch.exp(z - m), 0.0)
        total = torch.where(live[:, None], ez.sum(dim=1, keepdim=True), 1.0)
        p = ez / total
        top = z.sort(dim=1, descending=True, stable=True)
        ok = live[:, None] & (top.values[:, :K] > -math.inf)
        at = top.indices[:, :K]
        w = torch.where(ok, p.gather(1, at), 0.0)
        kept = w.sum(dim=1, keepdim=True)
        kept = torch.where(kept > 0, kept, 1.0)
        if s["normalize"]:
            w = w / kept
        hits = torch.zeros(T, E, device=z.device).scatter_(1, at, ok.float())
        counts, n = hits.sum(dim=0, dtype=torch.float64), live.sum()
        nf = n.clamp(min=1).float()
        load = (counts / counts.sum().clamp(min=1)).float()
        importance = p.sum(dim=0) / nf
        lse = torch.where(live, m[:, 0] + torch.log(total[:, 0]), 0.0)
        loss = torch.stack([E * (load * importance).sum(), (lse * lse).sum() / nf])
        out = {"ids": torch.where(ok, at, -1).to(I32), "weights": w, "counts": torch.cat([counts, n[None]]).to(I32), "load": load,
               "importance": importance, "loss": loss}
        if s["form"] == "train":
            gw = torch.where(ok, s["grad_weights"], 0.0)
            if s["normalize"]:
                gw = torch.where(ok, (gw - (gw * w).sum(dim=1, keepdim=True)) / kept, 0.0)
            gp = (BALANCE * E / nf * load)[None, :].expand(T, E).scatter_add(1, at, gw)
            inner = (gp * p).sum(dim=1, keepdim=True)
            out["grad_logits"] = (p * (gp - inner + 2 * ZLOSS / nf * lse[:, None])).to(s["logits"].dtype)
        return out
    if op == "dispatch":
        offsets, place = _plan(s["ids"], s["experts"])
        T, D, K = s["tokens"], s["dim"], s["top"]
        rows = torch.zeros(T * K + 1, D, device=place.device, dtype=s["x"].dtype)
        at = place.flatten().long()
        rows[torch.where(at >= 0, at, T * K)] = s["x"][:, None, :].expand(T, K, D).reshape(T * K, D)
        return {"offsets": offsets, "place": place, "rows": rows[:-1]}
    if op == "combine":
        T, K, D, dt = s["tokens"], s["top"], s["dim"], s["rows"].dtype
        ok = s["place"] >= 0
        at = torch.where(ok, s["place"], 0).long()
        w = torch.where(ok, s["weights"], 0.0)
        mine = s["rows"][at].float()
        out = {"out": (mine * w[:, :, None]).sum(dim=1).to(dt)}
        if s["form"] == "train":
            dy = s["grad_out"].float()
            out["grad_weights"] = torch.where(ok, (mine * dy[:, None, :]).sum(dim=2), 0.0)
            grad = torch.zeros(T * K + 1, D, device=dy.device, dtype=dt)
            grad[torch.where(ok, at, T * K).flatten()] = (w[:, :, None] * dy[:, None, :]).to(dt).view(T * K, D)
            out["grad_rows"] = grad[:-1]
        return out
    if op == "experts":
        # every active expert's rows padded to the most of one, in one batched product
        active, R = s["active"], s["x"].shape[0]
        first, past = s["offsets"][:-1][active].long(), s["offsets"][1:][active].long()
        at = first[:, None] + torch.arange(s["most"], device=first.device)
        ok = at < past[:, None]
        at = torch.where(ok, at, R)

        def spread(t):
            return torch.cat([t, torch.zeros_like(t[:1])])[at]

        def collect(t, dtype=BF16):
            flat = torch.zeros(R + 1, t.shape[-1], device=t.device, dtype=dtype)
            flat[at.flatten()] = t.to(dtype).flatten(0, 1)
            return flat[:-1]

        x = spread(s["x"].float())
        wg, wu, wd = (s[k][active].float() for k in ("wg", "wu", "wd"))
        g, u = x @ wg.transpose(1, 2), x @ wu.transpose(1, 2)
        y = collect((_act(g, s["act"])[0] * u) @ wd.transpose(1, 2))
        if s["form"] == "forward":
            return {"out": y}
        x, g, u = _eight_bits(x), _eight_bits(g), _eight_bits(u)
        a, da = _act(g, s["act"])
        dy = spread(s["dy"].float())
        dh = dy @ wd
        dg, du = dh * u * da, dh * a
        out = {"out": y, "dx": collect(dg @ wg + du @ wu)}
        for name, grad in (("dwg", dg.transpose(1, 2) @ x), ("dwu", du.transpose(1, 2) @ x), ("dwd", dy.transpose(1, 2) @ (a * u))):
            out[name] = torch.zeros_like(s[name])
            out[name][active] = grad.to(BF16)
        return out
    return {"back": _eight_bits(s["x"].float()).to(s["x"].dtype)}


def work(case):
    op = case["op"]
    e = 2 if case.get("dtype") == "bf16" else 4
    if op == "route":
        T, E, K = case["tokens"], case["experts"], case["top"]
        forward = T * E * e + T * (K * 8 + 5) + E * 12
        if case["form"] == "loss":
            return {"bytes": forward, "flops": 6 * T * E}
        return {"bytes": forward + T * E * e + T * K * 4, "flops": 12 * T * E}
    if op in ("dispatch", "combine"):
        T, D, K = case["tokens"], case["dim"], case["top"]
        if op == "dispatch":
            return {"bytes": T * K * 8 + (T + T * K) * D * e, "flops": T * K}
        forward = T * K * 8 + (T + T * K) * D * e
        if case["form"] == "forward":
            return {"bytes": forward, "flops": 2 * T * K * D}
        return {"bytes": forward + T * K * 4 + (T + T * K) * D * e, "flops": 5 * T * K * D}
    if op == "experts":
        D, F, E, R = case["dim"], case["ffn"], case["experts"], case["tokens"] * case["top"]
        weights = 3 * min(E, R) * D * F * 2  # of the experts that can have rows
        if case["form"] == "forward":
            return {"bytes": weights + 2 * R * D * 2, "flops": 6 * R * D * F}
        return {"bytes": weights + 3 * E * D * F * 2 + 4 * R * D * 2, "flops": 18 * R * D * F}
    n = case["rows"] * case["cols"]
    return {"bytes": 2 * n * e + 2 * (n + n // BLOCK), "flops": 4 * n}


def _steps64(x):
    """The 8-bit values of x in 64 bits: a block's step is the least power of two that is no less than largest / 127."""
    R, C = x.shape
    out = torch.zeros(R, -(-C // BLOCK) * BLOCK, device=x.device, dtype=torch.float64)
    out[:, :C] = x
    blocks = out.view(R, -1, BLOCK)
    largest = blocks.abs().max(dim=2, keepdim=True).values
    fraction, exponent = torch.frexp(largest / 127)  # fraction 0.5: a power of two itself
    step = torch.pow(2.0, (exponent - fraction.eq(0.5).int()).to(torch.float64))
    return (torch.round(blocks / step) * step).view(R, -1)[:, :C]


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "route":
        T, E, K = case["tokens"], case["experts"], case["top"]
        z = s["logits"].to(f64)
        dead = torch.isneginf(z).all(dim=1) | (s["valid"] == 0)
        z = z.masked_fill(dead[:, None], 0.0).requires_grad_()
        n = max(1, T - int(dead.sum()))
        alive = (~dead).to(f64)
        logp = torch.log_softmax(z, dim=1)
        p = logp.exp() * alive[:, None]
        lse = torch.logsumexp(z, dim=1) * alive
        chosen = torch.sort(s["logits"].to(f64), dim=1, descending=True, stable=True).indices[:, :K]
        w = p.gather(1, chosen)
        if case["normalize"]:
            w = w / w.sum(dim=1, keepdim=True).masked_fill(dead[:, None], 1.0)
        counts = torch.bincount(chosen[~dead].flatten(), minlength=E)
        load = counts.to(f64) / max(1, int(counts.sum()))
        importance = p.sum(dim=0) / n
        balance, zloss = E * torch.dot(load, importance), lse.square().sum() / n
        ids = chosen.masked_fill(dead[:, None], -1).to(I32)
        out = {"ids": ids, "weights": w.detach(), "counts": torch.cat([counts, counts.new_tensor([T - int(dead.sum())])]).to(I32), "load": load,
               "importance": importance.detach(), "loss": torch.stack([balance, zloss]).detach()}
        if case["form"] == "train":
            total = BALANCE * balance + ZLOSS * zloss + (w * s["grad_weights"].to(f64) * alive[:, None]).sum()
            out["grad_logits"] = torch.autograd.grad(total, z)[0]
        return out
    if op == "dispatch":
        ids = s["ids"].cpu().numpy().reshape(-1)
        T, K, E = case["tokens"], case["top"], case["experts"]
        order = sorted((i for i in range(T * K) if ids[i] >= 0), key=lambda i: int(ids[i]))  # a stable sort
        place = torch.full((T * K,), -1, dtype=torch.int64)
        place[torch.tensor(order, dtype=torch.int64)] = torch.arange(len(order))
        starts = [0] * (E + 1)
        for i in order:
            starts[int(ids[i]) + 1] += 1
        offsets = torch.tensor(starts).cumsum(0)
        rows = torch.zeros(T * K, case["dim"], device=DEV, dtype=f64)
        rows[:len(order)] = s["x"].to(f64)[torch.tensor(order, device=DEV, dtype=torch.int64) // K]
        return {"offsets": offsets.to(I32), "place": place.to(I32).view(T, K), "rows": rows}
    if op == "combine":
        K = case["top"]
        keep = s["place"].ge(0).to(f64)
        rows = s["rows"].to(f64)
        index = s["place"].clamp(min=0).long()
        out = torch.zeros(case["tokens"], case["dim"], device=DEV, dtype=f64)
        for k in range(K):
            out += (s["weights"][:, k].to(f64) * keep[:, k])[:, None] * rows.index_select(0, index[:, k])
        if case["form"] == "forward":
            return {"out": out}
        dy = s["grad_out"].to(f64)
        grad_rows, grad_weights = torch.zeros_like(rows), torch.zeros_like(keep)
        for k in range(K):
            grad_weights[:, k] = torch.linalg.vecdot(rows.index_select(0, index[:, k]), dy) * keep[:, k]
            grad_rows.index_add_(0, index[:, k], (s["weights"][:, k].to(f64) * keep[:, k])[:, None] * dy)
        return {"out": out, "grad_rows": grad_rows, "grad_weights": grad_weights}
    if op == "experts":
        bounds = s["offsets"].tolist()
        train = case["form"] == "train"
        y = torch.zeros(s["x"].shape, device=DEV, dtype=f64)
        dx = torch.zeros_like(y)
        grads = {k: torch.zeros(s[k].shape, device=DEV, dtype=f64) for k in (("dwg", "dwu", "dwd") if train else ())}
        lin = torch.nn.functional.linear
        for e in range(case["experts"]):
            rows = slice(bounds[e], bounds[e + 1])
            if rows.start == rows.stop:
                continue
            x, wg, wu, wd = s["x"][rows].to(f64), s["wg"][e].to(f64), s["wu"][e].to(f64), s["wd"][e].to(f64)

            def hidden(g, u):
                return (torch.nn.functional.silu(g) if case["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")) * u
            g, u = lin(x, wg), lin(x, wu)
            y[rows] = lin(hidden(g, u), wd)
            if train:
                x, g, u = _steps64(x), _steps64(g).requires_grad_(), _steps64(u).requires_grad_()
                h, dy = hidden(g, u), s["dy"][rows].to(f64)
                dg, du = torch.autograd.grad(h, (g, u), dy @ wd)
                dx[rows] = dg @ wg + du @ wu
                grads["dwg"][e], grads["dwu"][e], grads["dwd"][e] = dg.T @ x, du.T @ x, dy.T @ h.detach()
        return {"out": y, "dx": dx, **grads} if train else {"out": y}
    return {"back": _steps64(s["x"].to(f64))}
