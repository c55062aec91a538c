"""The dense operators around the expert stage, with their plain forms, as cases to be timed and compared.

  norm      residual addition, root-mean-square norm, and its rounding to 8 bits: e4m3 with a scale for each 128
            values of a row (the projections' input), or q8_1 blocks (the latent D projection's input)
  quantize  rounding of rows to e4m3 with a scale for each 128 values
  dense     y = x w^T for e4m3 rows (a scale for each 128 values of a row) and e4m3 weights (a scale for each
            128 x 128 block)
  ffn       the gated feed-forward block in the same format: silu(x gate^T) * (x up^T), rounded to e4m3 rows again,
            and the down projection

`own` chooses between the plain forms (elementary torch operations) and the framework's calls.
"""
import math

import torch

own = False

BLOCK = 128                  # values with one scale
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126      # smallest scale of a block
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # the norm before a decode step's projections: four tokens of a 4096-wide model
        {"name": "norm decode", "op": "norm", "T": 4, "C": 4096, "x": "bf16", "residual": "bf16", "y": "none", "out": "fp8"},
        # the latent layer's norm: the expert stage's fp32 rows added to a bf16 residual stream, q8_1 rows out
        {"name": "norm latent q8_1", "op": "norm", "T": 5268, "C": 4096, "x": "f32", "residual": "bf16", "y": "none", "out": "q8_1"},
        # a long prompt's norm: e4m3 rows for the projections, bf16 rows for the router's logits
        {"name": "norm prompt", "op": "norm", "T": 21000, "C": 4096, "x": "bf16", "residual": "bf16", "y": "bf16", "out": "fp8"},
        # rows that no norm precedes (an attention output), a ragged last block
        {"name": "quantize ragged", "op": "quantize", "T": 333, "C": 2000, "x": "f16"},
        {"name": "quantize prompt", "op": "quantize", "T": 21000, "C": 4096, "x": "bf16"},
        # the latent U projection of one decode step
        {"name": "dense decode", "op": "dense", "T": 4, "N": 4096, "K": 1024, "y": "f32"},
        # a chunk of a prompt, odd in every direction
        {"name": "dense odd chunk", "op": "dense", "T": 517, "N": 4100, "K": 2064, "y": "bf16"},
        # the latent D projection of a prompt
        {"name": "dense latent D", "op": "dense", "T": 5268, "N": 1024, "K": 4096, "y": "f32"},
        # a hidden-to-hidden projection of a long prompt
        {"name": "dense long prompt", "op": "dense", "T": 21000, "N": 4096, "K": 4096, "y": "bf16"},
        # a shared expert beside the routed ones: decode, and a prompt chunk; then a dense layer's wide block
        {"name": "ffn decode", "op": "ffn", "T": 4, "C": 4096, "F": 2048},
        {"name": "ffn chunk", "op": "ffn", "T": 512, "C": 4096, "F": 2048},
        {"name": "ffn wide prompt", "op": "ffn", "T": 5268, "C": 4096, "F": 8192},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["norm", "quantize", "dense", "dense", "ffn"])
    T = _log_int(rng, 1, 21000)
    if op == "norm":
        out = rng.choice(["fp8", "fp8", "q8_1"])
        return {"op": op, "T": T, "C": _log_int(rng, 256, 4096, 32), "x": rng.choice(["f32", "bf16", "f16"]),
                "residual": rng.choice(["f32", "bf16", "f16", "none"]), "y": rng.choice(["f32", "bf16", "none"]), "out": out}
    if op == "quantize":
        return {"op": op, "T": T, "C": _log_int(rng, 128, 4096, 16), "x": rng.choice(["f32", "bf16", "f16"])}
    if op == "dense":
        return {"op": op, "T": T, "N": _log_int(rng, 8, 4096), "K": _log_int(rng, 128, 4096, 16), "y": rng.choice(["f32", "bf16"])}
    return {"op": op, "T": _log_int(rng, 1, 5268), "C": _log_int(rng, 256, 4096, 16), "F": _log_int(rng, 128, 8192, 16)}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _quantize(v):
    """fp32 rows -> (e4m3 codes, scales), a scale for each 128 values of a row."""
    T, C = v.shape
    nb = _blocks(C)
    p = torch.zeros(T, nb * BLOCK, device=v.device)
    p[:, :C] = v
    p = p.view(T, nb, BLOCK)
    d = (p.abs().amax(2) / E4M3_MAX).clamp_min(SCALE_MIN)
    codes = (p * (1.0 / d)[..., None]).view(T, nb * BLOCK)[:, :C].to(torch.float8_e4m3fn)
    return codes.contiguous(), d


def _dequantize(codes, scales):
    """e4m3 rows with a scale for each 128 values -> fp32."""
    return codes.float() * scales.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _dequantize_weight(codes, scales):
    """e4m3 matrix with a scale for each 128 x 128 block -> fp32."""
    s = scales.repeat_interleave(BLOCK, 0)[:codes.shape[0]].repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.float() * s


def _weight(g, N, K, gain):
    """A weight matrix in e4m3: Gaussian entries whose size differs from block to block."""
    nn, nk = _blocks(N), _blocks(K)
    spread = torch.exp(0.5 * torch.randn(nn, nk, generator=g, device="cuda"))
    w = torch.zeros(nn * BLOCK, nk * BLOCK, device="cuda")
    w[:N, :K] = torch.randn(N, K, generator=g, device="cuda") * (gain / math.sqrt(K))
    b = w.view(nn, BLOCK, nk, BLOCK).mul_(spread[:, None, :, None])
    d = (b.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(SCALE_MIN)
    codes = (b / d[:, None, :, None]).view(nn * BLOCK, nk * BLOCK)[:N, :K].to(torch.float8_e4m3fn)
    return codes.contiguous(), d


def _rows(g, T, C, dtype=torch.float32):
    """Activation rows: some channels are larger than the rest, and rows differ in size."""
    channel = torch.exp(0.7 * torch.randn(1, C, generator=g, device="cuda"))
    row = torch.exp(0.3 * torch.randn(T, 1, generator=g, device="cuda"))
    return (torch.randn(T, C, generator=g, device="cuda") * channel * row).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]
    s = {"case": case}
    if op == "norm":
        C = case["C"]
        s["x"] = _rows(g, T, C, TYPES[case["x"]])
        s["weight"] = 1.0 + 0.2 * torch.randn(C, generator=g, device="cuda")
        s["residual"] = s["residual_out"] = s["y"] = None
        if case["residual"] != "none":
            s["residual"] = _rows(g, T, C, TYPES[case["residual"]])
            s["residual_out"] = torch.empty_like(s["residual"])
        if case["y"] != "none":
            s["y"] = torch.empty(T, C, dtype=TYPES[case["y"]], device="cuda")
        if case["out"] == "fp8":
            s["codes"] = torch.empty(T, C, dtype=torch.float8_e4m3fn, device="cuda")
            s["scales"] = torch.empty(T, _blocks(C), device="cuda")
        else:
            s["q8_1"] = torch.empty(T, C // 32, 36, dtype=torch.uint8, device="cuda")
    elif op == "quantize":
        C = case["C"]
        s["x"] = _rows(g, T, C, TYPES[case["x"]])
        s["codes"] = torch.empty(T, C, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(T, _blocks(C), device="cuda")
    elif op == "dense":
        N, K = case["N"], case["K"]
        s["x"], s["xs"] = _quantize(_rows(g, T, K))
        s["w"], s["ws"] = _weight(g, N, K, 1.0)
        s["y"] = torch.empty(T, N, dtype=TYPES[case["y"]], device="cuda")
    else:
        C, F = case["C"], case["F"]
        s["x"], s["xs"] = _quantize(_rows(g, T, C))
        gate, gate_s = _weight(g, F, C, 1.0)
        up, up_s = _weight(g, F, C, 1.0)
        # one matrix: the gate rows, then the up rows; each half has its own scale blocks
        s["gateup"], s["gateup_s"] = torch.cat([gate.view(torch.uint8), up.view(torch.uint8)]).view(torch.float8_e4m3fn), torch.stack([gate_s, up_s])
        s["down"], s["down_s"] = _weight(g, C, F, 1.0)
        s["y"] = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
        # memory for the intermediate rows, as much as any form of the block needs
        s["workspace"] = torch.empty(5 * T * F + (16 << 20), dtype=torch.uint8, device="cuda")
    return s


def _run_norm(s):
    case = s["case"]
    fp8 = case["out"] == "fp8"
    if own:
        import quantized_latent_moe_amd as lm
        lm.rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"], y=s["y"],
                   y_q8_1=None if fp8 else s["q8_1"], y_fp8=s["codes"] if fp8 else None, y_scales=s["scales"] if fp8 else None)
        out = {"residual": s["residual_out"], "y": s["y"]}
        if fp8:
            out.update(codes=s["codes"], scales=s["scales"])
        else:  # the values that the blocks stand for: fp16 d times the int8 codes
            b = s["q8_1"]
            out["values"] = b[:, :, 0:2].view(torch.float16) * b[:, :, 4:].view(torch.int8)
    else:
        v = s["x"].float()
        out = {"residual": None, "y": None}
        if s["residual"] is not None:
            v = v + s["residual"].float()
            out["residual"] = v.to(s["residual"].dtype)
        # the mean square in 64 bits: the codes next to a border between two codes depend on it
        r = torch.rsqrt(v.double().square().mean(1, keepdim=True) + EPS).float()
        y = v * r * s["weight"]
        if case["y"] != "none":
            out["y"] = y.to(TYPES[case["y"]])
        if fp8:
            out["codes"], out["scales"] = _quantize(y)
        else:
            b = y.view(case["T"], case["C"] // 32, 32)
            d = b.abs().amax(2, keepdim=True) / 127.0
            q = b * torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
            q = torch.trunc(q + torch.copysign(torch.full_like(q, 0.49999997), q))  # half away from zero
            out["values"] = d.half() * q.to(torch.int8)
    return {k: v for k, v in out.items() if v is not None}


def _run_quantize(s):
    if own:
        import quantized_latent_moe_amd as lm
        lm.quantize_fp8(s["x"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    codes, scales = _quantize(s["x"].float())
    return {"codes": codes, "scales": scales}


def _run_dense(s):
    if own:
        import quantized_latent_moe_amd as lm
        bf16 = s["case"]["y"] == "bf16"
        lm.dense_fp8(s["x"], s["xs"], s["w"], s["ws"], y_f32=None if bf16 else s["y"], y_bf16=s["y"] if bf16 else None)
        return s["y"]
    y = _dequantize(s["x"], s["xs"]) @ _dequantize_weight(s["w"], s["ws"]).t()
    return y.to(TYPES[s["case"]["y"]])


def _run_ffn(s):
    if own:
        import quantized_latent_moe_amd as lm
        lm.ffn_fp8(s["x"], s["xs"], s["gateup"], s["gateup_s"], s["down"], s["down_s"], s["workspace"], y_bf16=s["y"])
        return s["y"]
    F = s["case"]["F"]
    x = _dequantize(s["x"], s["xs"])
    gate = x @ _dequantize_weight(s["gateup"][:F], s["gateup_s"][0]).t()
    up = x @ _dequantize_weight(s["gateup"][F:], s["gateup_s"][1]).t()
    codes, scales = _quantize(gate / (1.0 + torch.exp(-gate)) * up)
    return (_dequantize(codes, scales) @ _dequantize_weight(s["down"], s["down_s"]).t()).to(torch.bfloat16)


def run(state):
    return {"norm": _run_norm, "quantize": _run_quantize, "dense": _run_dense, "ffn": _run_ffn}[state["case"]["op"]](state)


def work(case):
    op, T = case["op"], case["T"]
    size = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
    if op == "norm":
        C = case["C"]
        out = C + 4 * _blocks(C) if case["out"] == "fp8" else C // 32 * 36
        return {"bytes": T * (C * (size[case["x"]] + 2 * size[case["residual"]] + size[case["y"]]) + out) + 4 * C, "flops": 8 * T * C}
    if op == "quantize":
        C = case["C"]
        return {"bytes": T * (C * size[case["x"]] + C + 4 * _blocks(C)), "flops": 3 * T * C}
    if op == "dense":
        N, K = case["N"], case["K"]
        return {"bytes": T * (K + 4 * _blocks(K)) + N * K + 4 * _blocks(N) * _blocks(K) + T * N * size[case["y"]], "flops": 2 * T * N * K}
    C, F = case["C"], case["F"]
    return {"bytes": T * (C + 4 * _blocks(C)) + 3 * C * F + 12 * _blocks(C) * _blocks(F) + 2 * T * C, "flops": 6 * T * C * F}


# ---- the definitions in 64 bits ----

def _e4m3_64(v):
    """The nearest e4m3 value, ties to even, of 64-bit numbers within +-448."""
    _, e = torch.frexp(v)                                   # |v| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _blocked_64(v):
    T, C = v.shape
    nb = _blocks(C)
    return torch.nn.functional.pad(v, (0, nb * BLOCK - C)).view(T, nb, BLOCK)


def _quantize_64(v):
    b = _blocked_64(v)
    d = torch.clamp(b.abs().amax(2) / E4M3_MAX, min=SCALE_MIN)
    return _e4m3_64((b / d[..., None]).reshape(v.shape[0], -1)[:, :v.shape[1]]), d


def _rows_64(codes, scales):
    k = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return codes.double() * scales.double()[:, k]


def _weight_64(codes, scales):
    n = torch.arange(codes.shape[0], device=codes.device) // BLOCK
    k = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return codes.double() * scales.double()[n][:, k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["x"].double()
        out = {}
        if s["residual"] is not None:
            v = v + s["residual"].double()
            out["residual"] = v
        y = v / torch.sqrt((v * v).sum(1, keepdim=True) / case["C"] + EPS) * s["weight"].double()
        if case["y"] != "none":
            out["y"] = y
        if case["out"] == "fp8":
            out["codes"], out["scales"] = _quantize_64(y)
        else:
            b = y.view(case["T"], case["C"] // 32, 32)
            d = b.abs().amax(2, keepdim=True) / 127.0
            q = b / torch.where(d > 0, d, torch.ones_like(d))
            out["values"] = torch.sign(q) * torch.floor(q.abs() + 0.5) * d
        return out
    if op == "quantize":
        codes, scales = _quantize_64(s["x"].double())
        return {"codes": codes, "scales": scales}
    if op == "dense":
        return _rows_64(s["x"], s["xs"]) @ _weight_64(s["w"], s["ws"]).t()
    F = case["F"]
    x = _rows_64(s["x"], s["xs"])
    gate = x @ _weight_64(s["gateup"][:F], s["gateup_s"][0]).t()
    up = x @ _weight_64(s["gateup"][F:], s["gateup_s"][1]).t()
    codes, scales = _quantize_64(gate * torch.sigmoid(gate) * up)
    return (codes * scales.repeat_interleave(BLOCK, 1)[:, :F]) @ _weight_64(s["down"], s["down_s"]).t()
