"""Cases of a general router and of 8-bit linear layers for experts, in plain torch operations and as calls of the library.

Operators (``op`` of a case):
  route           scores of the experts (softmax or sigmoid), a bias for balance, groups of experts, the top k, their weights
  route_backward  the weights' gradient back to the logits
  quant           values into e4m3 with a scale for each 128 of a row, or for each 128 x 128 block of weights, and the
                  same transposed (the layout in which the gradients' products contract)
  linear          products of such rows with the weights of one layer, or, block by block of a plan, of its experts
  linear_dw       the gradient of those weights, summed over the layer's or each expert's rows

Scales are fp32 (amax / 448), or e8m0 (the power of two at or above that).  A plan groups the routes by expert and pads
each group to ``block_m`` rows.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    def route(name, op, T, E, top_k, scoring, groups, elem, **more):
        c = dict(name=name, op=op, T=T, E=E, top_k=top_k, scoring=scoring, elem=elem, bias=groups > 1, n_group=groups,
                 topk_group=max(1, groups // 2), group_top=2 if groups > 1 else 1, renorm=True, scale=2.5, masked=False)
        return {**c, **more}

    return [
        # one decode step of eight sequences: latency
        route("route-decode", "route", 8, 256, 8, "sigmoid", 8, "f32"),
        # a long prefill or a training micro-batch
        route("route-prefill", "route", 8192, 288, 8, "sigmoid", 8, "f32"),
        # the router's gradient of a small batch, weights not renormalised: every logit has a gradient
        route("route-backward-softmax", "route_backward", 64, 256, 6, "softmax", 1, "bf16", renorm=False, scale=1.0),
        # a training micro-batch's gradient
        route("route-backward", "route_backward", 8192, 288, 8, "sigmoid", 8, "f32"),
        # the activations of a decode step
        dict(name="quant-decode", op="quant", form="rows", M=32, N=0, K=4096, elem="bf16", scale="f32"),
        # a micro-batch's activations, kept for the forward and transposed for the weights' gradient
        dict(name="quant-train", op="quant", form="both", M=8192, N=0, K=4096, elem="bf16", scale="e8m0"),
        # the weights of eight experts after an optimizer step, for the forward and transposed for the backward
        dict(name="quant-weights", op="quant", form="weights", M=8, N=4096, K=4096, elem="f32", scale="f32"),
        # one token through a shared expert's gate and up projections
        dict(name="linear-1", op="linear", T=1, K=7168, N=4096, E=1, top_k=0, block_m=0, scale="f32", elem="bf16"),
        # a long prefill through the same layer
        dict(name="linear-prefill", op="linear", T=8192, K=7168, N=4096, E=1, top_k=0, block_m=0, scale="e8m0", elem="bf16"),
        # the experts of one of eight devices, on the routes of a prefill
        dict(name="linear-experts", op="linear", T=2048, K=4096, N=4096, E=32, top_k=8, block_m=128, scale="f32", elem="bf16"),
        # weights' gradient of a dense layer and of experts, for a training micro-batch
        dict(name="dw-dense", op="linear_dw", T=8192, K=4096, N=4096, E=1, top_k=0, block_m=0, scale="e8m0", elem="bf16"),
        dict(name="dw-experts", op="linear_dw", T=2048, K=4096, N=2048, E=32, top_k=6, block_m=128, scale="f32", elem="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route_backward", "quant", "linear", "linear", "linear_dw"))
    if op in ("route", "route_backward"):
        groups = rng.choice((1, 1, 4, 8))
        E = groups * max(2, _log(rng, 8, 512) // groups)
        half = max(1, groups // 2)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, top_k=min(rng.randint(1, 10), half * (E // groups)),
                    scoring=rng.choice(("softmax", "sigmoid")), elem=rng.choice(("f32", "f32", "bf16", "f16")),
                    bias=rng.random() < 0.6, n_group=groups, topk_group=half, group_top=rng.choice((1, 2)),
                    renorm=rng.random() < 0.6, scale=rng.choice((1.0, 2.5)), masked=rng.random() < 0.3)
    scale = rng.choice(("f32", "e8m0"))
    if op == "quant":
        form = rng.choice(("rows", "rows", "columns", "both", "weights"))
        c = dict(op=op, form=form, M=_log(rng, 1, 8192), N=0, K=16 * _log(rng, 4, 256),
                 elem=rng.choice(("bf16", "bf16", "f16", "f32")), scale=scale)
        return {**c, "M": rng.randint(1, 4), "N": 16 * _log(rng, 4, 256)} if form == "weights" else c
    c = dict(op=op, T=_log(rng, 1, 4096), K=16 * _log(rng, 16, 384), N=16 * _log(rng, 8, 256), E=1, top_k=0, block_m=0,
             scale=scale, elem=rng.choice(("bf16", "bf16", "f16")))
    if op == "linear" and rng.random() < 0.3:
        c["N"] += rng.randint(1, 15)
    if rng.random() < 0.5:
        E, top_k = _log(rng, 4, 32), rng.randint(1, 4)
        T = _log(rng, 1, 2048)
        per = T * top_k / E
        block_m = 16 if per < 8 else 32 if per < 24 else 64 if per < 64 else 128 if per < 256 else 256
        c.update(T=T, E=E, top_k=top_k, K=min(c["K"], 4096), N=min(c["N"], 2048),
                 block_m=max(128, block_m) if op == "linear_dw" else block_m)
    return c


# ---- inputs ----------------------------------------------------------------

def _plan(ids, E, block_m):
    """Route ids grouped by expert and padded to block_m with -1, the blocks' experts, and the row count."""
    flat = ids.reshape(-1).long()
    R = flat.numel()
    cap = R + min(E, R) * (block_m - 1)
    blocks = -(-cap // block_m)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + block_m - 1) // block_m * block_m
    first, start = torch.cumsum(counts, 0) - counts, torch.cumsum(padded, 0) - padded
    e = flat[order]
    plan = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    plan[start[e] + torch.arange(R, device="cuda") - first[e]] = order.int()
    ntp = padded.sum()
    at = torch.arange(blocks, device="cuda") * block_m
    of = torch.searchsorted(torch.cumsum(padded, 0), at, right=True)
    return plan, torch.where(at < ntp, of, -1).int(), ntp.int().reshape(1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, s = case, {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if c["op"] in ("route", "route_backward"):
        T, E, k = c["T"], c["E"], c["top_k"]
        logits = randn(T, E) * 2.0
        if c["masked"]:  # experts that a token may not use; the last token may use none
            logits[torch.rand(T, E, generator=g, device="cuda") < 0.2] = -math.inf
            logits[-1] = -math.inf
        s["logits"] = logits.to(TYPES[c["elem"]])
        s["bias"] = randn(E) * 0.1 if c["bias"] else None
        s["ids"], w = _route(s, c)
        s["dw"] = randn(T, k)
        s["out"] = (torch.empty_like(s["ids"]), torch.empty_like(w)) if c["op"] == "route" else torch.empty_like(s["logits"])
        return s
    if c["op"] == "quant":
        if c["form"] == "weights":
            s["x"] = (randn(c["M"], c["N"], c["K"]) / math.sqrt(c["K"])).to(TYPES[c["elem"]])
        else:
            s["x"] = (randn(c["M"], c["K"]) * torch.exp(randn(c["M"], 1))).to(TYPES[c["elem"]])
        s["out"] = tuple(None if v is None else torch.empty_like(v) for v in _quant(s["x"], c))
        return s
    T, K, N, E, k = c["T"], c["K"], c["N"], c["E"], c["top_k"]
    M, live = T, None
    s["experts"] = s["ntp"] = None
    if k:
        ids = torch.topk(torch.rand(T, E, generator=g, device="cuda"), k, dim=1)[1]
        plan, s["experts"], s["ntp"] = _plan(ids, E, c["block_m"])
        M, live = plan.numel(), (plan >= 0)[:, None]

    def rows(n, token):
        v = randn(T, n) if token or not k else randn(M, n)
        if token and k:
            v = v[(plan.clamp(min=0) // k).long()]
        return v if live is None else torch.where(live, v, 0.0)  # nothing in the padding rows

    if c["op"] == "linear":
        s["x"], s["x_scale"] = _quant_rows(rows(K, True), c["scale"])
        w = torch.empty(E, N, K, dtype=E4M3, device="cuda")
        parts = []
        for e in range(E):
            w[e], p = _quant_blocks(randn(N, K) / math.sqrt(K), c["scale"])
            parts.append(p)
        s["w"], s["w_scale"] = w, torch.stack(parts)
        s["out"] = torch.zeros(M, N, dtype=TYPES[c["elem"]], device="cuda")
        return s
    s["dyt"], s["dyt_scale"] = _quant_rows(_columns(rows(N, False) * 0.01), c["scale"])
    s["xt"], s["xt_scale"] = _quant_rows(_columns(rows(K, True)), c["scale"])
    s["out"] = torch.empty(E, N, K, dtype=TYPES[c["elem"]], device="cuda")
    return s


# ---- plain forms -----------------------------------------------------------

def _scores(logits, scoring):
    """In 64 bits, since two scores on either side of the choice may lie that near; 0 for a masked expert."""
    v = logits.double()
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    top = v.amax(1, keepdim=True)
    p = torch.exp(v - torch.where(torch.isinf(top), 0.0, top))
    return p / p.sum(1, keepdim=True).clamp(min=1e-300)


def _route(s, c):
    T, E, k, G = c["T"], c["E"], c["top_k"], c["n_group"]
    score = _scores(s["logits"], c["scoring"])
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(torch.isinf(s["logits"]), -math.inf, choice)
    if G > 1:
        best = torch.topk(choice.reshape(T, G, -1), c["group_top"], dim=2)[0]
        total = torch.where(torch.isinf(best), 0.0, best).sum(2)
        total = torch.where(torch.isinf(best[:, :, 0]), -math.inf, total)
        keep = torch.sort(total, dim=1, descending=True, stable=True)[1][:, :c["topk_group"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=total.device).scatter_(1, keep, True)
        choice = torch.where(kept.repeat_interleave(E // G, 1), choice, -math.inf)
    top, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    none = torch.isinf(top[:, :k])
    w = torch.where(none, 0.0, score.gather(1, ids[:, :k]))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(none, -1, ids[:, :k]).int(), (w * c["scale"]).float()


def _route_backward(s, c):
    score, ids = _scores(s["logits"], c["scoring"]), s["ids"].long()
    live = ids >= 0
    ids = ids.clamp(min=0)
    dw = torch.where(live, s["dw"].double(), 0.0) * c["scale"]
    p = torch.where(live, score.gather(1, ids), 0.0)
    if c["renorm"]:
        total = p.sum(1, keepdim=True).clamp(min=1e-300)
        dw = (dw - (p / total * dw).sum(1, keepdim=True)) / total
    d = torch.zeros_like(score).scatter_add_(1, ids, torch.where(live, dw, 0.0))
    if c["scoring"] == "sigmoid":
        d = d * score * (1.0 - score)
    else:
        d = score * (d - (d * score).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _power(e):
    """2^e in 64 bits, exactly (torch's pow and ldexp on the GPU are not)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale(amax, kind):
    """A group's scale as it is held, and its inverse."""
    amax = amax.clamp(min=1e-30)
    if kind == "f32":
        scale = amax * (1.0 / 448.0)
        return scale, 1.0 / scale
    m, x = torch.frexp(amax)  # m in [0.5, 1): 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875)
    return (e + 127).to(torch.uint8), _power(-e).float()


def _padded(v, dims):
    """Zeros behind the values, up to whole groups of 128."""
    pads = [0, -v.shape[-1] % 128] + ([0, -v.shape[-2] % 128] if dims == 2 else [])
    return torch.nn.functional.pad(v, pads)


def _quant_rows(x, kind):
    K = x.shape[-1]
    v = _padded(x.float(), 1)
    v = v.reshape(*v.shape[:-1], -1, 128)
    scale, inv = _scale(v.abs().amax(-1), kind)
    return (v * inv[..., None]).flatten(-2)[..., :K].contiguous().to(E4M3), scale


def _quant_blocks(w, kind):
    N, K = w.shape[-2:]
    v = _padded(w.float(), 2)
    v = v.reshape(*v.shape[:-2], v.shape[-2] // 128, 128, v.shape[-1] // 128, 128)
    scale, inv = _scale(v.abs().amax((-3, -1)), kind)
    q = (v * inv[..., :, None, :, None]).flatten(-4, -3).flatten(-2)
    return q[..., :N, :K].contiguous().to(E4M3), scale


def _columns(x):
    """The columns as rows, their length whole groups of 128."""
    return _padded(x.transpose(-1, -2), 1)


def _quant(x, c):
    if c["form"] == "weights":
        q, s = _quant_blocks(x, c["scale"])
        return q, s, q.transpose(1, 2).contiguous(), s.transpose(1, 2).contiguous()
    rows = _quant_rows(x, c["scale"]) if c["form"] in ("rows", "both") else (None, None)
    cols = _quant_rows(_columns(x), c["scale"]) if c["form"] in ("columns", "both") else (None, None)
    return rows + cols


def _scale_value(s, like):
    if s.dtype == torch.uint8:
        return torch.where(s == 255, math.nan, _power(s.long() - 127)).to(like)
    return s.to(like)


def _values(q, s, like=torch.float32):
    """What rows of codes and their scales stand for."""
    return q.to(like) * _scale_value(s, like).repeat_interleave(128, -1)[..., :q.shape[-1]]


def _block_values(q, s):
    f = _scale_value(s, torch.float32).repeat_interleave(128, -1)[..., :q.shape[-1]]
    return q.float() * f.repeat_interleave(128, -2)[..., :q.shape[-2], :]


def _linear(s, c):
    x = _values(s["x"], s["x_scale"])
    if s["experts"] is None:
        return torch.matmul(x, _block_values(s["w"][0], s["w_scale"][0]).t()).to(TYPES[c["elem"]])
    M, bm = x.shape[0], c["block_m"]
    blocks = s["experts"].numel()
    x = torch.nn.functional.pad(x, [0, 0, 0, blocks * bm - M]).reshape(blocks, bm, -1)
    w = _block_values(s["w"], s["w_scale"])[s["experts"].clamp(min=0).long()]
    y = torch.matmul(x, w.transpose(1, 2)).reshape(blocks * bm, -1)[:M]
    return torch.where(torch.arange(M, device=y.device)[:, None] < s["ntp"], y, 0.0).to(TYPES[c["elem"]])


def _linear_dw(s, c):
    dy, x = _values(s["dyt"], s["dyt_scale"]), _values(s["xt"], s["xt_scale"])
    if s["experts"] is None:
        return torch.matmul(dy, x.t())[None].to(TYPES[c["elem"]])
    bm, blocks = c["block_m"], s["experts"].numel()
    pad = [0, max(0, blocks * bm - x.shape[1])]

    def cut(v):
        return torch.nn.functional.pad(v, pad)[:, :blocks * bm].reshape(-1, blocks, bm).transpose(0, 1)

    parts = torch.matmul(cut(dy), cut(x).transpose(1, 2))
    at = torch.where(s["experts"] < 0, c["E"], s["experts"]).long()
    out = torch.zeros(c["E"] + 1, *parts.shape[1:], device=x.device).index_add_(0, at, parts)
    return out[:c["E"]].to(TYPES[c["elem"]])


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import mixture_experts_ffn_moe_amd as moe
        if op == "route":
            ids, w = moe.moe_route_topk(s["logits"], c["top_k"], s["bias"], c["scoring"], c["n_group"], c["topk_group"],
                                        c["group_top"], c["renorm"], c["scale"], out=s["out"])
            return {"ids": ids, "weights": w}
        if op == "route_backward":
            return moe.moe_route_topk_backward(s["logits"], s["ids"], s["dw"], c["scoring"], c["renorm"], c["scale"],
                                               out=s["out"])
        if op == "quant":
            if c["form"] == "weights":
                got = moe.moe_fp8_quant_weights(s["x"], c["scale"], transposed=True, out=s["out"])
            else:
                got = moe.moe_fp8_quant(s["x"], c["scale"], rows=c["form"] != "columns", columns=c["form"] != "rows",
                                        out=s["out"])
            return dict(zip(("q", "scale", "qt", "scale_t"), got))
        if op == "linear":
            return moe.moe_fp8_linear(s["x"], s["x_scale"], s["w"], s["w_scale"], s["experts"], s["ntp"], c["block_m"],
                                      out=s["out"])
        return moe.moe_fp8_linear_dw(s["dyt"], s["dyt_scale"], s["xt"], s["xt_scale"], c["E"], s["experts"], s["ntp"],
                                     c["block_m"], out=s["out"])
    if op == "route":
        ids, w = _route(s, c)
        return {"ids": ids, "weights": w}
    if op == "route_backward":
        return _route_backward(s, c)
    if op == "quant":
        return dict(zip(("q", "scale", "qt", "scale_t"), _quant(s["x"], c)))
    return _linear(s, c) if op == "linear" else _linear_dw(s, c)


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    c, op = case, case["op"]
    es = 4 if c["elem"] == "f32" else 2
    if op in ("route", "route_backward"):
        T, E, k = c["T"], c["E"], c["top_k"]
        if op == "route":
            return {"bytes": T * (E * es + 8 * k), "flops": 4 * T * E}
        dense = c["scoring"] == "softmax" and not c["renorm"]  # else the selected logits alone are read
        return {"bytes": T * (E * es * (2 if dense else 1) + (8 + (0 if dense else es)) * k), "flops": 4 * T * k}
    scale = 4 if c["scale"] == "f32" else 1
    if op == "quant":
        if c["form"] == "weights":
            n = c["M"] * c["N"] * c["K"]
            return {"bytes": n * (es + 2) + 2 * scale * n // 16384, "flops": 2 * n}
        n, copies = c["M"] * c["K"], 2 if c["form"] == "both" else 1
        return {"bytes": n * (es + copies) + copies * scale * n // 128, "flops": 2 * n * copies}
    T, K, N, E, k = c["T"], c["K"], c["N"], c["E"], c["top_k"]
    rows, active = T, 1
    if k:
        active = E * (1 - (1 - k / E) ** T)
        rows = T * k
    if op == "linear":
        return {"bytes": rows * K * (1 + scale / 128) + active * N * K + 2 * rows * N, "flops": 2 * rows * N * K}
    return {"bytes": rows * (N + K) * (1 + scale / 128) + 2 * E * N * K, "flops": 2 * rows * N * K}


# ---- in 64 bits, from the definitions --------------------------------------

def _exact_quant(v, kind):
    """The nearest e4m3 values of the rows of v, each a group, and the groups' scales."""
    amax = v.abs().amax(1, keepdim=True).clamp(min=1e-30)
    scale = amax / 448
    if kind != "f32":
        m, x = torch.frexp(scale)
        scale = _power(x - (m == 0.5).int())
    y = v / scale
    step = _power(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)  # four significant bits
    return torch.round(y / step) * step, scale[:, 0]


def _exact_rows(x, kind):
    M, K = x.shape
    q = torch.zeros(M, K, dtype=torch.float64, device=x.device)
    s = torch.zeros(M, -(-K // 128), dtype=torch.float64, device=x.device)
    for j in range(s.shape[1]):
        q[:, j * 128:j * 128 + 128], s[:, j] = _exact_quant(x[:, j * 128:j * 128 + 128], kind)
    return q, s


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "route":
        ids, rows = s["ids"].long(), torch.arange(c["T"], device="cuda")
        v = s["logits"].double()
        if c["scoring"] == "sigmoid":
            p = torch.sigmoid(v)
        else:
            p = torch.nan_to_num(torch.softmax(v, 1))
        w = torch.zeros(c["T"], c["top_k"], dtype=torch.float64, device="cuda")
        for j in range(c["top_k"]):
            w[:, j] = p[rows, ids[:, j].clamp(min=0)] * (ids[:, j] >= 0)
        total = w.sum(1)
        if c["renorm"]:
            w = w / torch.where(total > 0, total, 1.0)[:, None]
        return {"ids": None, "weights": w * c["scale"]}
    if op == "route_backward":
        v = s["logits"].double().requires_grad_()
        with torch.enable_grad():
            if c["scoring"] == "sigmoid":
                p = torch.sigmoid(v)
            else:
                p = torch.softmax(torch.where(torch.isinf(v).all(1, keepdim=True), torch.zeros_like(v), v), 1)
            w = p.gather(1, s["ids"].long().clamp(min=0)) * (s["ids"] >= 0)
            if c["renorm"]:
                w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
            (w * c["scale"] * s["dw"].double()).sum().backward()
        return v.grad
    if op == "quant":
        x = s["x"].double()
        if c["form"] == "weights":
            q, qt = torch.empty_like(x), torch.empty_like(x.transpose(1, 2))
            nb, kb = -(-c["N"] // 128), -(-c["K"] // 128)
            sc = torch.empty(c["M"], nb, kb, dtype=torch.float64, device="cuda")
            for i in range(nb):
                for j in range(kb):
                    part = x[:, i * 128:i * 128 + 128, j * 128:j * 128 + 128]
                    y, sc[:, i, j] = _exact_quant(part.reshape(c["M"], -1), c["scale"])
                    q[:, i * 128:i * 128 + 128, j * 128:j * 128 + 128] = y.reshape(part.shape)
            qt.copy_(q.transpose(1, 2))
            got = (q, sc, qt, sc.transpose(1, 2).contiguous())
        else:
            rows = _exact_rows(x, c["scale"]) if c["form"] != "columns" else (None, None)
            cols = (None, None)
            if c["form"] != "rows":
                xt = torch.zeros(c["K"], -(-c["M"] // 128) * 128, dtype=torch.float64, device="cuda")
                xt[:, :c["M"]] = x.t()
                cols = _exact_rows(xt, c["scale"])
            got = rows + cols
        if c["scale"] == "e8m0":  # whole numbers: compared as such
            got = (got[0], None, got[2], None)
        return dict(zip(("q", "scale", "qt", "scale_t"), got))
    if op == "linear":
        x = _values(s["x"], s["x_scale"], torch.float64)

        def weight(e):
            f = _scale_value(s["w_scale"][e], torch.float64)
            n, k = torch.arange(c["N"], device="cuda") // 128, torch.arange(c["K"], device="cuda") // 128
            return s["w"][e].double() * f[n][:, k]

        if s["experts"] is None:
            return x @ weight(0).t()
        out = torch.zeros(x.shape[0], c["N"], dtype=torch.float64, device="cuda")
        of = s["experts"].repeat_interleave(c["block_m"])[:x.shape[0]]
        for e in range(c["E"]):
            at = torch.nonzero(of == e)[:, 0]
            out[at] = x[at] @ weight(e).t()
        return out
    dy, x = _values(s["dyt"], s["dyt_scale"], torch.float64), _values(s["xt"], s["xt_scale"], torch.float64)
    if s["experts"] is None:
        return (dy @ x.t())[None]
    out = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device="cuda")
    of = s["experts"].repeat_interleave(c["block_m"])
    for e in range(c["E"]):
        at = torch.nonzero(of == e)[:, 0]
        out[e] = dy[:, at] @ x[:, at].t()
    return out
