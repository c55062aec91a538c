"""The 16-bit products and the routing rules around the expert stage, with their plain forms, as cases to be timed and
compared.

  dense   y = act(x w^T + bias) + residual for rows and weights in bf16 or fp16; y in fp32, bf16, fp16, or as q8_1
          blocks (the expert stage's latent rows)
  gated   act(x gate^T + bias) * (x up^T + bias), the first half of a gated feed-forward block in the same types
  router  softmax or sigmoid scores, a bias for balance, groups of experts, top-k, renormalised and scaled weights

`own` chooses between the plain forms (elementary torch operations) and the framework's calls.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LOWEST = torch.finfo(torch.float32).min


def listed():
    return [
        # the router's logits of one decode step: four tokens of a 4096-wide model, 128 experts
        {"name": "dense logits decode", "op": "dense", "T": 4, "N": 128, "K": 4096, "type": "bf16", "y": "f32", "bias": False, "act": "none", "residual": "none", "slice": False},
        # a projection of one decode step, added to the residual stream
        {"name": "dense decode", "op": "dense", "T": 4, "N": 4096, "K": 4096, "type": "bf16", "y": "bf16", "bias": False, "act": "none", "residual": "bf16", "slice": False},
        # a chunk of a prompt, odd in every direction, its rows a slice of wider ones
        {"name": "dense odd chunk", "op": "dense", "T": 517, "N": 4100, "K": 2056, "type": "f16", "y": "f16", "bias": True, "act": "gelu", "residual": "f32", "slice": True},
        # the router's logits of a prompt
        {"name": "dense logits prompt", "op": "dense", "T": 5268, "N": 128, "K": 4096, "type": "bf16", "y": "f32", "bias": True, "act": "none", "residual": "none", "slice": False},
        # the latent D projection of a prompt, rounded to the expert stage's rows
        {"name": "dense latent D q8_1", "op": "dense", "T": 5268, "N": 1024, "K": 4096, "type": "bf16", "y": "q8_1", "bias": False, "act": "none", "residual": "none", "slice": False},
        # a hidden-to-hidden projection of a long prompt, added to the residual stream
        {"name": "dense long prompt", "op": "dense", "T": 21000, "N": 4096, "K": 4096, "type": "bf16", "y": "bf16", "bias": False, "act": "none", "residual": "bf16", "slice": False},
        # a shared expert beside the routed ones: decode, and a prompt chunk; then a dense layer's wide block
        {"name": "gated decode", "op": "gated", "T": 4, "K": 4096, "F": 2048, "type": "bf16", "y": "bf16", "bias": False, "act": "silu"},
        {"name": "gated chunk", "op": "gated", "T": 512, "K": 4096, "F": 2048, "type": "f16", "y": "f16", "bias": True, "act": "gelu_tanh"},
        {"name": "gated wide prompt", "op": "gated", "T": 5268, "K": 4096, "F": 8192, "type": "bf16", "y": "bf16", "bias": False, "act": "silu"},
        # one decode step's routing with a balance bias and groups
        {"name": "router decode", "op": "router", "T": 4, "E": 128, "k": 8, "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_score": "top2", "renormalise": True, "scale": 2.5, "masked": 0},
        # a prompt's routing by biased softmax scores over all experts
        {"name": "router prompt", "op": "router", "T": 5268, "E": 128, "k": 8, "score": "softmax", "bias": True, "groups": 1, "top_groups": 1, "group_score": "max", "renormalise": True, "scale": 1.0, "masked": 0},
        # a long prompt's routing over many experts in groups, some of them closed
        {"name": "router long prompt", "op": "router", "T": 21000, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_score": "top2", "renormalise": True, "scale": 2.5, "masked": 8},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["dense", "dense", "gated", "router"])
    T = _log_int(rng, 1, 21000)
    if op == "router":
        E = rng.choice([8, 16, 24, 60, 64, 96, 128, 160, 192, 256])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        return {"op": op, "T": T, "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.7, "groups": groups, "top_groups": top_groups,
                "group_score": rng.choice(["max", "top2"]), "renormalise": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0, 0, 3])}
    kind, K = rng.choice(["bf16", "bf16", "f16"]), _log_int(rng, 64, 8192, 8)
    bias, act = rng.random() < 0.5, rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
    if op == "dense":
        y = rng.choice(["f32", kind, kind, "q8_1"])
        N = _log_int(rng, 32, 8192, 32) if y == "q8_1" else _log_int(rng, 8, 8192)
        T = min(T, 21000 * 4096 * 4096 // (N * K))
        return {"op": op, "T": T, "N": N, "K": K, "type": kind, "y": y, "bias": bias, "act": act, "residual": rng.choice(["none", "f32", kind]), "slice": rng.random() < 0.3}
    F = _log_int(rng, 16, 8192)
    T = min(T, 21000 * 4096 * 2048 // (F * K))
    return {"op": op, "T": T, "K": K, "F": F, "type": kind, "y": rng.choice(["f32", kind, kind]), "bias": bias, "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh"])}


def _rows(g, T, C):
    """Activation rows: some channels are larger than the rest, and rows differ in size."""
    channel = torch.exp(0.7 * torch.randn(1, C, generator=g, device="cuda"))
    row = torch.exp(0.3 * torch.randn(T, 1, generator=g, device="cuda"))
    return torch.randn(T, C, generator=g, device="cuda") * channel * row


def _weight(g, N, K):
    return torch.randn(N, K, generator=g, device="cuda") * K ** -0.5


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]
    s = {"case": case, "bias": None, "residual": None}
    if op == "router":
        E = case["E"]
        rank = torch.argsort(torch.rand(E, generator=g, device="cuda"))
        # some experts are more popular than others; closed ones have -inf
        s["logits"] = torch.randn(T, E, generator=g, device="cuda") - 0.3 * torch.log1p(rank.float())
        s["logits"][:, rank >= E - case["masked"]] = -math.inf
        if case["bias"]:
            s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda")
        s["idx"] = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(T, case["k"], device="cuda")
        return s
    kind, K, N = TYPES[case["type"]], case["K"], case["N"] if op == "dense" else case["F"]
    if case.get("slice"):
        s["x"] = _rows(g, T, 2 * K).to(kind)[:, K:]
    else:
        s["x"] = _rows(g, T, K).to(kind)
    s["w"] = _weight(g, N if op == "dense" else 2 * N, K).to(kind)
    if case["bias"]:
        s["bias"] = 0.5 * torch.randn(s["w"].shape[0], generator=g, device="cuda")
    if op == "dense" and case["residual"] != "none":
        s["residual"] = _rows(g, T, N).to(TYPES[case["residual"]])
    if case["y"] == "q8_1":
        s["y"] = torch.empty(T, N // 32, 36, dtype=torch.uint8, device="cuda")
    else:
        s["y"] = torch.empty(T, N, dtype=TYPES[case["y"]], device="cuda")
    return s


def _activate(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _run_dense(s):
    case = s["case"]
    q8 = case["y"] == "q8_1"
    if own:
        import quantized_latent_moe_amd as lm
        lm.dense_16(s["x"], s["w"], bias=s["bias"], activation=case["act"], residual=s["residual"],
                    y=None if q8 else s["y"], y_q8_1=s["y"] if q8 else None)
        if q8:  # the values that the blocks stand for: fp16 d times the int8 codes
            b = s["y"]
            return b[:, :, 0:2].view(torch.float16) * b[:, :, 4:].view(torch.int8)
        return s["y"]
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _activate(v, case["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    if not q8:
        return v.to(TYPES[case["y"]])
    b = v.view(case["T"], case["N"] // 32, 32)
    d = b.abs().amax(2, keepdim=True) / 127.0
    q = b * torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    q = torch.trunc(q + torch.copysign(torch.full_like(q, 0.49999997), q))  # half away from zero
    return d.half() * q.to(torch.int8)


def _run_gated(s):
    case = s["case"]
    if own:
        import quantized_latent_moe_amd as lm
        lm.gated_16(s["x"], s["w"], s["y"], bias=s["bias"], activation=case["act"])
        return s["y"]
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    F = case["F"]
    return (_activate(v[:, :F], case["act"]) * v[:, F:]).to(TYPES[case["y"]])


def _run_router(s):
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    if own:
        import quantized_latent_moe_amd as lm
        lm.router_topk_ex(s["logits"], k, s["idx"], s["w"], bias=s["bias"], score=case["score"], groups=G,
                          top_groups=case["top_groups"], group_score=case["group_score"], renormalise=case["renormalise"],
                          scale=case["scale"])
        return {"idx": s["idx"], "w": s["w"]}
    # scores in 64 bits, rounded once: the order of near ones depends on it
    v = s["logits"].double()
    if case["score"] == "softmax":
        p = torch.exp(v - v.amax(1, keepdim=True))
        p = (p / p.sum(1, keepdim=True)).float()
    else:
        p = (1.0 / (1.0 + torch.exp(-v))).float()
    c = p if s["bias"] is None else p + s["bias"]
    closed = s["logits"] == -math.inf
    c = torch.where(closed, torch.full_like(c, LOWEST), c)
    if G > 1:
        top = torch.sort(c.view(T, G, E // G), dim=2, descending=True)[0]
        score = top[:, :, 0]
        if case["group_score"] == "top2":
            score = score + torch.where(top[:, :, 1] > LOWEST, top[:, :, 1], torch.zeros_like(score))
        kept = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        inside = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        c = torch.where(inside.repeat_interleave(E // G, 1), c, torch.full_like(c, -math.inf))
    idx = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.where(closed, torch.zeros_like(p), p).gather(1, idx).double()
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.to(torch.int32), "w": (w * case["scale"]).float()}


def run(state):
    return {"dense": _run_dense, "gated": _run_gated, "router": _run_router}[state["case"]["op"]](state)


def work(case):
    op, T = case["op"], case["T"]
    size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
    if op == "router":
        return {"bytes": 4 * T * case["E"] + 4 * case["E"] * case["bias"] + 8 * T * case["k"], "flops": 20 * T * case["E"]}
    K = case["K"]
    if op == "gated":
        F = case["F"]
        return {"bytes": 2 * T * K + 4 * F * K + 8 * F * case["bias"] + T * F * size[case["y"]], "flops": 4 * T * F * K}
    N = case["N"]
    out = N // 32 * 36 if case["y"] == "q8_1" else N * size[case["y"]]
    return {"bytes": 2 * T * K + 2 * N * K + 4 * N * case["bias"] + T * (out + N * size[case["residual"]]), "flops": 2 * T * N * K}


# ---- the definitions in 64 bits ----

def _activate_64(v, act):
    if act == "relu":
        return v.clamp_min(0)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        # (1 + tanh(z)) / 2 is the logistic function of 2 z
        return v * torch.sigmoid(math.sqrt(8.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        v = s["logits"].double()
        p = torch.softmax(v, 1) if case["score"] == "softmax" else torch.sigmoid(v)
        # the ranking is defined on scores rounded to 32 bits; the weights are not
        c = p.float() if s["bias"] is None else p.float() + s["bias"]
        c = c.double().masked_fill(torch.isneginf(v), -1e30)
        if G > 1:
            a = c.reshape(T, G, E // G)
            first = a.max(2)
            score = first.values
            if case["group_score"] == "top2":
                second = a.scatter(2, first.indices[..., None], -2e30).amax(2)
                score = (score + torch.where(second > -1e29, second, 0.0)).float()
            order = torch.argsort(-score.double(), dim=1, stable=True)
            place = torch.argsort(order, dim=1)
            c = (a - 1e38 * (place >= case["top_groups"]).double()[..., None]).reshape(T, E)
        idx = torch.argsort(-c, dim=1, stable=True)[:, :k]
        w = p.gather(1, idx)
        if case["renormalise"]:
            w = w / w.sum(1, keepdim=True)
        return {"idx": idx.int(), "w": case["scale"] * w}
    v = torch.mm(s["x"].double(), s["w"].double().t().contiguous())
    if s["bias"] is not None:
        v += s["bias"].double()
    if op == "gated":
        gate, up = v.chunk(2, 1)
        return _activate_64(gate, case["act"]) * up
    v = _activate_64(v, case["act"])
    if s["residual"] is not None:
        v = v + s["residual"].double()
    if case["y"] != "q8_1":
        return v
    b = v.view(case["T"], -1, 32)
    d = b.abs().amax(2, keepdim=True) / 127.0
    q = b / torch.where(d > 0, d, torch.ones_like(d))
    return torch.sign(q) * torch.floor(q.abs() + 0.5) * d
