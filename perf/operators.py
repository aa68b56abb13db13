"""Cases, plain forms and exact values of the operators around the packed
ternary products: what stands between two of them in a decoder layer.

 - "norm":     RMSNorm of a product's output with the residual's addition, to
               fp32, bf16, or int8 with a scale per token (the input of the
               next int8 product).
 - "dispatch": a mixture-of-experts layer's tokens sorted by expert: the index
               arrays and the sorted rows.  "combine": the experts' rows back
               to their tokens, weighted.  "grad": the gradient of that in the
               rows and the weights.  "spread": the gradient of the sorting
               (the rows back to their tokens with weights of one).
 - "dense":    the product of int8 activations with a dense int8 weight, a
               scale per token and per output channel: the linears that stay
               dense (the output head, a router, attention projections).

`run` computes one pass, in plain torch operations, or, where `own` is true,
through the calls of `ternary_weight_amd.tq`.
"""
from __future__ import annotations

import math

import torch

own = False

F32, BF16, I8 = 0, 1, 2                    # the values of tq.F32, tq.BF16, tq.I8
TYPES = {F32: torch.float32, BF16: torch.bfloat16, I8: torch.int8}
SIZE = {F32: 4, BF16: 2, I8: 1}
EPS = 1e-5


def listed():
    return [
        # One token of a BitNet-2B-shaped decoder: the residual stream and a product's output, both fp32, to int8.
        {"name": "norm-decode", "op": "norm", "m": 1, "k": 2560, "x": F32, "res": True, "rt": F32, "y": I8},
        # Its FFN sub-norm over a 2048-token prompt: no residual there.
        {"name": "norm-ffn-prompt", "op": "norm", "m": 2048, "k": 6912, "x": F32, "res": False, "rt": F32, "y": I8},
        # A long batch of a 4096-wide model with a bf16 residual stream, an odd token count.
        {"name": "norm-bf16-long", "op": "norm", "m": 16381, "k": 4096, "x": BF16, "res": True, "rt": BF16, "y": BF16},
        # One decode batch of 64 tokens, 8 of 128 experts each, int8 rows with their scales.
        {"name": "dispatch-decode", "op": "dispatch", "t": 64, "top": 8, "e": 128, "h": 2048, "x": I8, "pad": 0.0},
        # A prompt batch in bf16 with padding tokens at its end, which go to no expert.
        {"name": "dispatch-prompt", "op": "dispatch", "t": 8192, "top": 8, "e": 128, "h": 2048, "x": BF16, "pad": 0.05},
        # The experts' fp32 outputs back to the decode batch.
        {"name": "combine-decode", "op": "combine", "t": 64, "top": 8, "e": 128, "h": 2048, "ys": F32, "y": F32, "pad": 0.0},
        # The same for the prompt batch, to a bf16 stream.
        {"name": "combine-prompt", "op": "combine", "t": 8192, "top": 8, "e": 128, "h": 2048, "ys": F32, "y": BF16, "pad": 0.05},
        # The gradient of a fine-tuning batch, an odd token count.
        {"name": "combine-grad", "op": "grad", "t": 4099, "top": 8, "e": 128, "h": 2048, "ys": BF16, "y": BF16, "pad": 0.0},
        # The output head at one token: a vocabulary of 128256 rows.
        {"name": "dense-head-decode", "op": "dense", "m": 1, "n": 128256, "k": 2560, "y": F32},
        # A few tokens against a deep weight.
        {"name": "dense-few", "op": "dense", "m": 13, "n": 4096, "k": 14336, "y": F32},
        # A prompt through a BitNet-2B-shaped gate.
        {"name": "dense-prompt", "op": "dense", "m": 2048, "n": 6912, "k": 2560, "y": F32},
        # A long batch through a Llama-8B-shaped gate, bf16 out.
        {"name": "dense-long", "op": "dense", "m": 8192, "n": 14336, "k": 4096, "y": BF16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dispatch", "combine", "grad", "spread", "dense", "dense", "dense"])
    if op == "norm":
        k = 16 * _log(rng, 8, 1024)
        return {"op": op, "m": _log(rng, 1, min(16381, 16381 * 4096 // k)), "k": k, "x": rng.choice([F32, BF16]),
                "res": rng.random() < 0.7, "rt": rng.choice([F32, BF16]), "y": rng.choice([F32, BF16, I8, I8])}
    if op == "dense":
        m, k = _log(rng, 1, 8192), 16 * _log(rng, 8, 896)
        n = _log(rng, 128, min(128256, 8192 * 14336 * 4096 // (m * k), 14336 * 8192 // m + 4096))
        return {"op": op, "m": m, "n": n, "k": k, "y": rng.choice([F32, BF16])}
    h, top = 16 * _log(rng, 16, 256), rng.randint(1, 8)
    c = {"op": op, "t": _log(rng, 1, min(8192, (4099 if op == "grad" else 8192) * 8 * 2048 // (top * h))),
         "top": top, "e": max(top, _log(rng, 4, 256)), "h": h, "pad": rng.choice([0.0, 0.0, 0.1, 0.3])}
    if op == "dispatch":
        c["x"] = rng.choice([F32, BF16, I8])
        if c["x"] == F32:                                  # as many bytes as the bf16 rows at most
            c["t"] = max(1, c["t"] // 2)
    else:
        c["ys"], c["y"] = rng.choice([F32, BF16]), rng.choice([F32, BF16])
        if op == "grad" and c["ys"] == F32:
            c["t"] = max(1, c["t"] // 2)
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _int8_rows(v):
    """int8 rows and their scales, as the per-token quantiser makes them."""
    a = v.abs().amax(1, keepdim=True).clamp_min(1e-30)
    return (v * (127.0 / a)).round().clamp(-127, 127).to(torch.int8), (a / 127.0).squeeze(1).contiguous()


def _route(g, t, top, e, pad):
    """Expert ids and weights of a router with uneven experts; the last `pad` of the tokens are padding (id -1)."""
    logits = _randn(g, t, e) + 0.7 * _randn(g, 1, e)
    top_logits, ids = logits.topk(top, dim=1)
    ids = ids.to(torch.int32)
    if int(pad * t):
        ids[t - int(pad * t):] = -1
    return ids.contiguous(), torch.softmax(top_logits, 1).contiguous()


def _typed(v, t):
    return v.to(TYPES[t]).contiguous()


def prepare(case, seed):
    g, s = _gen(seed), dict(case)
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        x = _randn(g, m, k) * (1.0 + 7.0 * (_rand(g, k) < 0.01))     # a few wide channels, as trained models have
        s["xv"] = _typed(x, case["x"])
        s["resv"] = _typed(2.0 * _randn(g, m, k), case["rt"]) if case["res"] else None
        s["w"] = 0.5 + _rand(g, k)
        s["hv"] = torch.empty(m, k, dtype=TYPES[case["rt"]], device="cuda") if case["res"] else None
        s["yv"] = torch.empty(m, k, dtype=TYPES[case["y"]], device="cuda")
        s["sv"] = torch.empty(m, device="cuda") if case["y"] == I8 else None
        s["vals"] = torch.empty(m, k, dtype=torch.bfloat16, device="cuda") if case["y"] == I8 else None
        return s
    if case["op"] == "dense":
        m, n, k = case["m"], case["n"], case["k"]
        s["xq"], s["xs"] = _int8_rows(_randn(g, m, k))
        s["wq"], s["ws"] = _int8_rows(_randn(g, n, k) * (0.02 * (0.5 + _rand(g, n, 1))))
        s["yv"] = torch.empty(m, n, dtype=TYPES[case["y"]], device="cuda")
        return s
    t, top, e, h = case["t"], case["top"], case["e"], case["h"]
    s["ids"], s["wts"] = _route(g, t, top, e, case["pad"])
    if case["op"] == "dispatch":
        x = _randn(g, t, h)
        s["xv"], s["xsc"] = _int8_rows(x) if case["x"] == I8 else (_typed(x, case["x"]), None)
        s["rows"] = torch.empty(t, top, dtype=torch.int32, device="cuda")
        s["pairs"] = torch.empty(t * top, dtype=torch.int32, device="cuda")
        s["offs"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
        s["out"] = torch.zeros(t * top, h, dtype=TYPES[case["x"]], device="cuda")   # rows behind the last expert stay
        s["outs"] = torch.zeros(t * top, device="cuda") if case["x"] == I8 else None
        return s
    s["rows"], _, _ = _plain_index(s["ids"], e)
    s["ysv"] = _typed(_randn(g, t * top, h), case["ys"])
    if case["op"] == "grad":
        s["dy"] = _typed(_randn(g, t, h), case["y"])
        s["dys"] = torch.zeros(t * top, h, dtype=TYPES[case["ys"]], device="cuda")
        s["dw"] = torch.empty(t, top, device="cuda")
    else:
        s["yv"] = torch.empty(t, h, dtype=TYPES[case["y"]], device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _plain_index(ids, e):
    """rows [t][top]: where each pair went; pairs: which pair each sorted row
    is; offsets: the experts' first rows.  Pairs of no expert get -1 and the
    rows behind the last expert hold no pair."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < e), flat, e)
    order = torch.sort(key, stable=True).indices
    n = flat.numel()
    place = torch.empty_like(order)
    place[order] = torch.arange(n, device=ids.device)
    rows = torch.where(key < e, place, -1).reshape(ids.shape).to(torch.int32)
    pairs = torch.where(key[order] < e, order, -1).to(torch.int32)
    counts = (key[:, None] == torch.arange(e, device=ids.device)).sum(0)
    offs = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return rows, pairs, offs


def _plain_norm(s):
    h = s["xv"].float()
    if s["res"]:
        h = h + s["resv"].float()
    mean = h.double().square().mean(1, keepdim=True).float()      # 64-bit sum: every later step is one fp32 rounding
    r = (mean + EPS).double().sqrt().float().double().reciprocal().float()
    n = (h * r) * s["w"]
    out = {"h": h.to(TYPES[s["rt"]])} if s["res"] else {}
    if s["y"] == I8:
        a = n.abs().amax(1, keepdim=True)
        inv = torch.where(a > 0, (127.0 / a.double()).float(), 0.0)
        q = (n * inv).round().clamp(-127, 127)
        scale = (a.double() / 127.0).float()
        return {**out, "y": (q * scale).to(torch.bfloat16), "scale": scale.squeeze(1)}
    return {**out, "y": n.to(TYPES[s["y"]])}


def _plain_dispatch(s):
    rows, pairs, offs = _plain_index(s["ids"], s["e"])
    used, token = pairs >= 0, pairs.clamp_min(0).long() // s["top"]
    out = {"rows": rows, "pairs": pairs, "offs": offs, "xs": torch.where(used[:, None], s["xv"][token], s["out"])}
    if s["x"] == I8:
        out["scale"] = torch.where(used, s["xsc"][token], s["outs"])
    return out


def _plain_combine(s):
    used = (s["rows"] >= 0)[..., None]
    v = s["ysv"][s["rows"].clamp_min(0).long()].float()
    if s["op"] == "combine":
        v = v * s["wts"][..., None]
    return {"y": torch.where(used, v, 0.0).sum(1).to(TYPES[s["y"]])}


def _plain_grad(s):
    used, at = s["rows"] >= 0, s["rows"].clamp_min(0).long()
    dy = s["dy"].float()[:, None, :]
    d_w = torch.where(used, (dy * s["ysv"][at].float()).sum(2), 0.0)
    n = s["dys"].shape[0]
    d_ys = torch.cat([s["dys"], s["dys"][:1]])                    # one row more, for the pairs of no expert
    d_ys[torch.where(used, at, n)] = (dy * s["wts"][..., None]).to(d_ys.dtype)
    return {"d_ys": d_ys[:n], "d_w": d_w}


def _plain_dense(s):
    acc = s["xq"].float() @ s["wq"].float().t()
    return {"y": (acc * (s["xs"][:, None] * s["ws"])).to(TYPES[s["y"]])}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from ternary_weight_amd import tq
    op = s["op"]
    if op == "norm":
        tq.rmsnorm(s["m"], s["k"], s["x"], s["xv"], s["w"], EPS, s["y"], s["yv"], s["sv"],
                   residual_type=s["rt"], residual=s["resv"], residual_out=s["hv"])
        out = {"h": s["hv"]} if s["res"] else {}
        if s["y"] == I8:                                   # the values that the int8 codes stand for
            return {**out, "y": torch.mul(s["yv"], s["sv"][:, None], out=s["vals"]), "scale": s["sv"]}
        return {**out, "y": s["yv"]}
    if op == "dispatch":
        if "ws" not in s:                                  # the program's workspace, kept from pass to pass
            s["ws"] = torch.empty(tq.moe_dispatch_workspace_size(s["t"], s["top"], s["e"]), dtype=torch.uint8,
                                  device="cuda")
        tq.moe_dispatch(s["t"], s["top"], s["e"], s["ids"], s["rows"], s["pairs"], s["offs"], s["h"], s["x"],
                        s["xv"], s["xsc"], s["out"], s["outs"], workspace=s["ws"], workspace_bytes=s["ws"].numel())
        out = {"rows": s["rows"], "pairs": s["pairs"], "offs": s["offs"], "xs": s["out"]}
        return {**out, "scale": s["outs"]} if s["x"] == I8 else out
    if op in ("combine", "spread"):
        tq.moe_combine(s["t"], s["top"], s["h"], s["t"] * s["top"], s["rows"], s["wts"] if op == "combine" else None,
                       s["ys"], s["ysv"], s["y"], s["yv"])
        return {"y": s["yv"]}
    if op == "grad":
        tq.moe_combine_grad(s["t"], s["top"], s["h"], s["t"] * s["top"], s["rows"], s["wts"], s["y"], s["dy"],
                            s["ys"], s["ysv"], s["dys"], s["dw"])
        return {"d_ys": s["dys"], "d_w": s["dw"]}
    tq.gemm_dense_i8(s["m"], s["n"], s["k"], s["xq"], s["xs"], s["wq"], s["ws"], s["y"], s["yv"])
    return {"y": s["yv"]}


PLAIN = {"norm": _plain_norm, "dispatch": _plain_dispatch, "combine": _plain_combine, "spread": _plain_combine,
         "grad": _plain_grad, "dense": _plain_dense}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


def work(case):
    op = case["op"]
    if op == "norm":
        m, k = case["m"], case["k"]
        each = SIZE[case["x"]] + (2 * SIZE[case["rt"]] if case["res"] else 0) + SIZE[case["y"]]
        return {"bytes": m * k * each + 4 * k + (4 * m if case["y"] == I8 else 0), "flops": 5 * m * k}
    if op == "dense":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * SIZE[case["y"]] + 4 * (m + n), "flops": 2 * m * n * k}
    t, top, h = case["t"], case["top"], case["h"]
    tokens = t - int(case["pad"] * t)
    pairs = tokens * top
    if op == "dispatch":
        row = h * SIZE[case["x"]] + (4 if case["x"] == I8 else 0)
        return {"bytes": 12 * t * top + 4 * (case["e"] + 1) + (tokens + pairs) * row, "flops": 0}
    if op == "grad":
        return {"bytes": 12 * t * top + tokens * h * SIZE[case["y"]] + 2 * pairs * h * SIZE[case["ys"]],
                "flops": 3 * pairs * h}
    return {"bytes": (8 if op == "combine" else 4) * t * top + pairs * h * SIZE[case["ys"]] + t * h * SIZE[case["y"]],
            "flops": (2 if op == "combine" else 1) * pairs * h}


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    """The definitions in 64 bits.  Whole numbers have none: the index arrays
    are compared by themselves, and int8 rows that are only moved too."""
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        h = s["xv"].double() + (s["resv"].double() if case["res"] else 0.0)
        n = s["w"].double() * h / ((h * h).sum(1, keepdim=True) / case["k"] + EPS).sqrt()
        out = {"h": h} if case["res"] else {}
        if case["y"] != I8:
            return {**out, "y": n}
        scale = n.abs().max(1, keepdim=True).values / 127
        step = torch.where(scale > 0, scale, 1.0)
        return {**out, "y": torch.round(n / step).clamp(-127, 127) * step, "scale": scale[:, 0]}
    if op == "dense":
        y = torch.empty(case["m"], case["n"], dtype=torch.float64, device="cuda")
        x = s["xq"].double() * s["xs"].double()[:, None]
        for a in range(0, case["n"], 16384):
            b = min(case["n"], a + 16384)
            y[:, a:b] = x @ (s["wq"][a:b].double() * s["ws"][a:b].double()[:, None]).t()
        return {"y": y}
    t, top = case["t"], case["top"]
    if op == "dispatch":
        xs, scale = s["out"].double(), None if case["x"] != I8 else s["outs"].double()
        flat, at = s["ids"].reshape(-1), 0
        for e in range(case["e"]):
            token = torch.nonzero(flat == e)[:, 0] // top
            xs[at:at + len(token)] = s["xv"][token].double()
            if scale is not None:
                scale[at:at + len(token)] = s["xsc"][token].double()
            at += len(token)
        none = {"rows": None, "pairs": None, "offs": None}
        return {**none, "xs": xs} if scale is None else {**none, "xs": None, "scale": scale}
    rows = s["rows"].long()
    if op == "grad":
        d_ys, d_w = s["dys"].double(), torch.zeros(t, top, dtype=torch.float64, device="cuda")
        for j in range(top):
            on = torch.nonzero(rows[:, j] >= 0)[:, 0]
            at = rows[on, j]
            d_ys[at] = s["dy"][on].double() * s["wts"][on, j].double()[:, None]
            d_w[on, j] = (s["dy"][on].double() * s["ysv"][at].double()).sum(1)
        return {"d_ys": d_ys, "d_w": d_w}
    y = torch.zeros(t, case["h"], dtype=torch.float64, device="cuda")
    for j in range(top):
        on = torch.nonzero(rows[:, j] >= 0)[:, 0]
        v = s["ysv"][rows[on, j]].double()
        y[on] += v * s["wts"][on, j].double()[:, None] if op == "combine" else v
    return {"y": y}
