"""Workloads of the 8-bit-integer operators: root-mean-square norm with the residual's addition and an int8 output,
row quantisation, the int8 product with token and channel scales, and the whole gated FFN over int8 weights.

Every case is a dict of plain values; prepare() makes what a program holds before the call, run() is one call.
With `own` true run() calls the package; otherwise it computes the same thing from elementary torch operations in
32 bits. exact() is the definition in 64 bits.

Int8 results are returned as the values they stand for (code times scale, in bfloat16)."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # the norm before an FFN, one token being decoded: latency
        {"name": "norm_decode_m1", "op": "norm", "M": 1, "K": 5120, "dtype": "bf16", "residual": True, "offset": 0.0},
        # a batch of uneven prompts, residual stream in 32 bits, weights stored as w - 1
        {"name": "norm_f32_m333", "op": "norm", "M": 333, "K": 5376, "dtype": "f32", "residual": True, "offset": 1.0},
        # a long prompt
        {"name": "norm_prefill_m8192", "op": "norm", "M": 8192, "K": 5120, "dtype": "bf16", "residual": True, "offset": 0.0},
        # the intermediate of three tokens under verification
        {"name": "quantize_f16_m3", "op": "quantize", "M": 3, "K": 17408, "dtype": "f16"},
        # a weight at load time
        {"name": "quantize_weight", "op": "quantize", "M": 17408, "K": 5120, "dtype": "bf16"},
        # one projection of one token: the weight is read once
        {"name": "gemm_decode_m1", "op": "gemm", "M": 1, "K": 5120, "N": 17408, "out": "bf16", "bias": False},
        # a ragged batch against an odd number of channels, 32-bit outputs
        {"name": "gemm_ragged_m300", "op": "gemm", "M": 300, "K": 4112, "N": 4099, "out": "f32", "bias": True},
        # one projection of a long prompt
        {"name": "gemm_prefill_m4096", "op": "gemm", "M": 4096, "K": 5120, "N": 17408, "out": "bf16", "bias": False},
        # the whole FFN: the smallest layer (latency of the call)
        {"name": "ffn_tiny_m1", "op": "ffn", "M": 1, "K": 256, "N": 512, "act": "silu", "out": "bf16"},
        # the whole FFN of one token
        {"name": "ffn_decode_m1", "op": "ffn", "M": 1, "K": 5120, "N": 17408, "act": "silu", "out": "bf16"},
        # the whole FFN of a batch of sequences being decoded together
        {"name": "ffn_batch_m32", "op": "ffn", "M": 32, "K": 5376, "N": 21504, "act": "gelu", "out": "bf16"},
        # the whole FFN of a prompt
        {"name": "ffn_prefill_m2048", "op": "ffn", "M": 2048, "K": 5120, "N": 17408, "act": "silu", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log16(rng, lo, hi):
    return max(lo, min(hi, _log(rng, lo, hi) // 16 * 16))


def draw(rng):
    op = rng.choice(["norm", "quantize", "gemm", "ffn"])
    if op in ("norm", "quantize"):
        K = _log16(rng, 256, 17408)
        most = (8192 if op == "norm" else 17408) * 5120
        c = {"op": op, "M": min(_log(rng, 1, 17408), max(1, most // (2 * K))), "K": K, "dtype": rng.choice(["bf16", "f16", "f32"])}
        if op == "norm":
            c["residual"] = rng.random() < 0.75
            c["offset"] = rng.choice([0.0, 1.0])
        return c
    K = _log16(rng, 256, 17408)
    if op == "gemm":
        N = min(_log(rng, 256, 21504), 17408 * 5120 // K)
        M = min(_log(rng, 1, 4096), 4096 * 5120 * 17408 // (N * K))
        return {"op": op, "M": M, "K": K, "N": N, "out": rng.choice(["bf16", "f16", "f32"]), "bias": rng.random() < 0.5}
    N = min(_log16(rng, 512, 21504), 5376 * 21504 // K // 16 * 16)
    M = min(_log(rng, 1, 2048), 2048 * 5120 * 17408 // (N * K))
    return {"op": op, "M": M, "K": K, "N": N, "act": rng.choice(["silu", "gelu"]), "out": rng.choice(["bf16", "f16"])}


def _weight(g, rows, cols):
    """Normal weights of a trained layer's size, as int8 codes with a scale for each row."""
    w = torch.randn(rows, cols, generator=g, device=DEV) / math.sqrt(cols)
    scales = w.abs().amax(1) / 127
    return (w / scales[:, None]).round_().to(torch.int8), scales


def _hidden(g, rows, cols):
    """A residual stream: a few channels far larger than the rest, tokens of unlike size."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.exp(torch.randn(rows, 1, generator=g, device=DEV) * 0.3)
    loud = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device=DEV)
    x[:, loud] *= 6.0
    return x


def _tokens(g, rows, cols):
    """Quantised activations: codes and a scale for each token."""
    x = _hidden(g, rows, cols)
    scales = x.abs().amax(1) / 127
    return (x / scales[:, None]).round_().to(torch.int8), scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        t = TYPES[case["dtype"]]
        s["x"] = (torch.randn(M, K, generator=g, device=DEV) * 0.5).to(t)
        s["r"] = _hidden(g, M, K).to(t) if case["residual"] else None
        s["w"] = (1.0 - case["offset"] + 0.2 * torch.randn(K, generator=g, device=DEV)).to(t)
    elif case["op"] == "quantize":
        s["x"] = _hidden(g, M, K).to(TYPES[case["dtype"]])
    elif case["op"] == "gemm":
        s["xc"], s["xs"] = _tokens(g, M, K)
        s["wc"], s["ws"] = _weight(g, case["N"], K)
        s["b"] = torch.randn(case["N"], generator=g, device=DEV) if case["bias"] else None
    else:
        s["xc"], s["xs"] = _tokens(g, M, K)
        s["gate"], s["up"] = _weight(g, case["N"], K), _weight(g, case["N"], K)
        s["down"] = _weight(g, K, case["N"])
    return s


# ---------------------------------------------------------------- plain forms, 32 bits


def _round8(y):
    """(codes as floats, scales) of the rows of y."""
    scales = y.abs().amax(1, keepdim=True) / 127
    inv = torch.where(scales > 0, 1 / scales, scales)
    return torch.round(y * inv).clamp(-127, 127), scales


def _values(codes, scales):
    """What codes and a scale for each row stand for."""
    out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    return torch.mul(codes, scales.view(-1, 1), out=out)


def _product(xc, xs, wc, ws):
    return (xc.float() @ wc.float().t()) * xs.view(-1, 1) * ws


def _gate(a, kind):
    if kind == "silu":
        return a * torch.sigmoid(a)
    return 0.5 * a * (1 + torch.tanh(0.7978845608028654 * (a + 0.044715 * a * a * a)))


def _plain(s):
    if s["op"] == "norm":
        v = s["x"].float()
        if s["r"] is not None:
            v = v + s["r"].float()
        y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * (s["w"].float() + s["offset"])
        codes, scales = _round8(y)
        out = {"values": _values(codes, scales), "scales": scales.view(-1)}
        if s["r"] is not None:
            out["sum"] = v.to(s["x"].dtype)
        return out
    if s["op"] == "quantize":
        codes, scales = _round8(s["x"].float())
        return {"values": _values(codes, scales), "scales": scales.view(-1)}
    if s["op"] == "gemm":
        y = _product(s["xc"], s["xs"], s["wc"], s["ws"])
        if s["b"] is not None:
            y = y + s["b"]
        return y.to(TYPES[s["out"]])
    h = _gate(_product(s["xc"], s["xs"], *s["gate"]), s["act"]) * _product(s["xc"], s["xs"], *s["up"])
    codes, scales = _round8(h)
    return _product(codes, scales, *s["down"]).to(TYPES[s["out"]])


def run(s):
    if not own:
        return _plain(s)
    import w4a16_nvfp4_dense_amd as ffn
    if s["op"] == "norm":
        codes, scales, total = ffn.int8_rmsnorm(s["x"], s["w"], EPS, residual=s["r"], weight_offset=s["offset"])
        out = {"values": _values(codes, scales), "scales": scales}
        if total is not None:
            out["sum"] = total
        return out
    if s["op"] == "quantize":
        codes, scales = ffn.int8_quantize(s["x"])
        return {"values": _values(codes, scales), "scales": scales}
    if s["op"] == "gemm":
        return ffn.int8_gemm(s["xc"], s["xs"], ffn.Int8DeviceWeight(s["wc"], s["ws"]), bias=s["b"], out_dtype=TYPES[s["out"]])
    act = ffn.ACT_SILU if s["act"] == "silu" else ffn.ACT_GELU_TANH
    return ffn.int8_forward(s["xc"], s["xs"], ffn.Int8DeviceWeight(*s["gate"]), ffn.Int8DeviceWeight(*s["up"]),
                            ffn.Int8DeviceWeight(*s["down"]), act, out_dtype=TYPES[s["out"]])


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        e = SIZE[case["dtype"]]
        moved = M * K * (e * (3 if case["residual"] else 1) + 1) + K * e + 4 * M
        return {"bytes": moved, "flops": 6 * M * K}
    if case["op"] == "quantize":
        return {"bytes": M * K * (SIZE[case["dtype"]] + 1) + 4 * M, "flops": 3 * M * K}
    N, e = case["N"], SIZE[case["out"]]
    if case["op"] == "gemm":
        return {"bytes": M * K + 4 * M + N * K + 4 * N * (2 if case["bias"] else 1) + M * N * e, "flops": 2 * M * N * K}
    return {"bytes": M * K + 4 * M + 3 * N * K + 4 * (2 * N + K) + M * K * e, "flops": 6 * M * N * K}


# ---------------------------------------------------------------- the definitions, 64 bits


def _steps(y):
    """Rows of y in whole steps of a 127th of their largest magnitude: (values, step)."""
    step = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 127.0
    q = (y / step.clamp_min(1e-300)[:, None]).round()
    return q * step[:, None], step


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "norm":
            v = s["x"].double()
            if s["r"] is not None:
                v = v.add(s["r"].double())
            ms = torch.linalg.vector_norm(v, dim=1).square() / case["K"]
            y = v / torch.sqrt(ms + EPS)[:, None] * s["w"].double().add(case["offset"])
            values, step = _steps(y)
            out = {"values": values, "scales": step}
            if s["r"] is not None:
                out["sum"] = v
            return out
        if case["op"] == "quantize":
            values, step = _steps(s["x"].double())
            return {"values": values, "scales": step}

        def real(codes, scales):
            return codes.double().mul_(scales.double()[:, None])

        def times(a, w):
            return torch.mm(a, real(*w).t())

        a = real(s["xc"], s["xs"])
        if case["op"] == "gemm":
            y = times(a, (s["wc"], s["ws"]))
            return y if s["b"] is None else y.add_(s["b"].double())
        g, u = times(a, s["gate"]), times(a, s["up"])
        if case["act"] == "silu":
            h = g / (1.0 + torch.exp(-g)) * u
        else:
            h = torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g.pow(3))) * g * u
        return times(_steps(h)[0], s["down"])
