"""Workloads of the sparse (mixture of experts) FFN's operators: the router's choice of experts, the plan that puts
the chosen (token, expert) pairs in expert order, the product grouped by expert over NVFP4 weights, and the whole
sparse gated FFN.

Every case is a dict of plain values; prepare() makes what a program holds before the call, run() is one call.
With `own` true run() calls the package; otherwise it computes the same thing from elementary torch operations in
32 bits (the keys that experts are chosen by, where a bias is added, in 64). exact() is the definition in 64 bits.

A chosen expert of -1 is no expert: padding tokens have such choices, and their outputs are zero."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
NVFP4_BYTES = 0.5 + 1 / 16  # of an element: its code and its share of a block scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the choice for one token being decoded: latency
        {"name": "route_decode_t1", "op": "route", "T": 1, "E": 64, "k": 8, "dtype": "bf16", "score": "softmax",
         "bias": False, "normalize": True, "scale": 1.0},
        # a batch of uneven prompts, each expert with a balancing bias that only the choice sees
        {"name": "route_sigmoid_t333", "op": "route", "T": 333, "E": 160, "k": 6, "dtype": "f32", "score": "sigmoid",
         "bias": True, "normalize": True, "scale": 2.5},
        # long prompts together
        {"name": "route_prefill_t16384", "op": "route", "T": 16384, "E": 256, "k": 8, "dtype": "bf16",
         "score": "softmax", "bias": False, "normalize": False, "scale": 1.0},
        # the expert order of sequences being decoded together
        {"name": "plan_batch_t32", "op": "plan", "T": 32, "E": 128, "k": 8, "pad": 3},
        # and of long prompts, the last ones' padding included
        {"name": "plan_prefill_t16384", "op": "plan", "T": 16384, "E": 256, "k": 8, "pad": 1000},
        # one projection of a few tokens each with an expert of its own: weights are read for a row or two
        {"name": "gemm_few_r64", "op": "gemm", "T": 64, "k": 1, "gather": False, "E": 64, "K": 2048, "N": 5120,
         "dtype": "bf16", "out": "bf16"},
        # an odd number of experts, rows and channels, 32-bit outputs
        {"name": "gemm_ragged_r777", "op": "gemm", "T": 259, "k": 3, "gather": True, "E": 17, "K": 4128, "N": 1999,
         "dtype": "f16", "out": "f32"},
        # one projection of a long prompt, its tokens' rows read where they are
        {"name": "gemm_prefill_r16384", "op": "gemm", "T": 4096, "k": 4, "gather": True, "E": 64, "K": 5120,
         "N": 2048, "dtype": "bf16", "out": "bf16"},
        # the whole FFN: the smallest layer (latency of the call)
        {"name": "ffn_tiny_t1", "op": "ffn", "T": 1, "E": 8, "k": 2, "K": 256, "N": 512, "act": "silu",
         "dtype": "bf16", "pad": 0},
        # the whole FFN of one token
        {"name": "ffn_decode_t1", "op": "ffn", "T": 1, "E": 64, "k": 8, "K": 5120, "N": 2048, "act": "silu",
         "dtype": "bf16", "pad": 0},
        # the whole FFN of a batch of sequences being decoded together, three of its places empty
        {"name": "ffn_batch_t32", "op": "ffn", "T": 32, "E": 128, "k": 8, "K": 2048, "N": 1024, "act": "gelu",
         "dtype": "f16", "pad": 3},
        # the whole FFN of a long prompt, padded to a round number of tokens
        {"name": "ffn_prefill_t4096", "op": "ffn", "T": 4096, "E": 64, "k": 8, "K": 5120, "N": 2048, "act": "silu",
         "dtype": "bf16", "pad": 77},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log32(rng, lo, hi):
    return max(lo, min(hi, _log(rng, lo, hi) // 32 * 32))


def draw(rng):
    op = rng.choice(["route", "plan", "gemm", "ffn"])
    if op in ("route", "plan"):
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        T = min(_log(rng, 1, 16384), 16384 * 256 // E)
        if op == "plan":
            return {"op": op, "T": T, "E": E, "k": k, "pad": rng.choice([0, T // 9])}
        c = {"op": op, "T": T, "E": E, "k": k, "dtype": rng.choice(["bf16", "f16", "f32"])}
        c["score"] = rng.choice(["softmax", "sigmoid"])
        c["bias"] = rng.random() < 0.5
        c["normalize"] = rng.random() < 0.5
        c["scale"] = rng.choice([1.0, 2.5])
        return c
    E = _log(rng, 4, 128)
    k = rng.randint(1, min(8, E))
    K = _log32(rng, 256, 5376)
    if op == "gemm":
        N = min(_log(rng, 128, 5376), 64 * 5120 * 2048 // (E * K))
        T = max(1, min(_log(rng, 1, 4096), 4096 * 4 * 5120 * 2048 // (k * N * K)))
        dtype = rng.choice(["bf16", "f16"])
        return {"op": op, "T": T, "k": k, "gather": rng.random() < 0.5, "E": E, "K": K, "N": N, "dtype": dtype,
                "out": rng.choice([dtype, "f32"])}
    N = max(32, min(_log32(rng, 128, 2048), 64 * 5120 * 2048 // (E * K) // 32 * 32))
    T = max(1, min(_log(rng, 1, 4096), 4096 * 8 * 5120 * 2048 // (k * N * K)))
    return {"op": op, "T": T, "E": E, "k": k, "K": K, "N": N, "act": rng.choice(["silu", "gelu"]),
            "dtype": rng.choice(["bf16", "f16"]), "pad": rng.choice([0, T // 9])}


def _logits(g, T, E):
    """A router's outputs: the tokens' own, and some experts a little more popular than others."""
    return torch.randn(T, E, generator=g, device=DEV) + 0.3 * torch.randn(E, generator=g, device=DEV)


def _choices(g, T, E, k, pad):
    """Chosen experts int32 [T, k] and their weights fp32 [T, k]; the last `pad` tokens have none."""
    p, ids = torch.topk(torch.softmax(_logits(g, T, E), 1), k, dim=1)
    p = p / p.sum(1, keepdim=True)
    ids = ids.to(torch.int32)
    if pad:
        ids[T - pad:] = -1
        p[T - pad:] = 0
    return ids, p


def _experts(g, E, rows, cols):
    """NVFP4 weights of E experts, from normal weights of a trained layer's size: codes [E, rows, cols/2] (the even
    column in the low half of a byte), E4M3 scales of 16 columns [E, rows, cols/16], an fp32 scale each [E]."""
    codes = torch.empty(E, rows, cols // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, rows, cols // 16, dtype=torch.uint8, device=DEV)
    scale2 = torch.empty(E, device=DEV)
    bounds = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device=DEV)
    for e in range(E):
        w = torch.randn(rows, cols // 16, 16, generator=g, device=DEV) / math.sqrt(cols)
        scale2[e] = w.abs().amax() / (6 * 448)
        block = (w.abs().amax(2) / (6 * scale2[e])).to(torch.float8_e4m3fn)
        scales[e] = block.view(torch.uint8)
        step = (block.float() * scale2[e]).clamp_min(1e-30).unsqueeze(2)
        q = torch.bucketize(w.abs() / step, bounds, out_int32=True).to(torch.uint8) | ((w < 0).to(torch.uint8) << 3)
        q = q.view(rows, cols)
        codes[e] = q[:, ::2] | (q[:, 1::2] << 4)
    return codes, scales, scale2


def _hidden(g, rows, cols):
    """Normed activations: a few channels far larger than the rest."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    loud = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device=DEV)
    x[:, loud] *= 6.0
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        s["logits"] = _logits(g, T, E).to(TYPES[case["dtype"]])
        s["b"] = 0.1 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        return s
    s["ids"], s["p"] = _choices(g, T, E, k, case.get("pad", 0))
    if case["op"] == "plan":
        return s
    t = TYPES[case["dtype"]]
    if case["op"] == "gemm":
        flat = s.pop("ids").view(-1)
        s["rows"] = torch.sort(flat, stable=True).indices.to(torch.int32) if case["gather"] else None
        s["offsets"] = torch.searchsorted(flat.sort().values, torch.arange(E + 1, device=DEV, dtype=torch.int32)).to(torch.int32)
        s["x"] = _hidden(g, T if case["gather"] else T * k, case["K"]).to(t)
        s["w"] = _experts(g, E, case["N"], case["K"])
    else:
        s["x"] = _hidden(g, T, case["K"]).to(t)
        s["gate"], s["up"] = _experts(g, E, case["N"], case["K"]), _experts(g, E, case["N"], case["K"])
        s["down"] = _experts(g, E, case["K"], case["N"])
    return s


# ---------------------------------------------------------------- plain forms, 32 bits


def _weight(w, e):
    """The weight of expert e in 32 bits, without its scale."""
    codes, scales, _ = w
    table = torch.tensor([*E2M1, *(-v for v in E2M1)], device=codes.device)
    c = codes[e].int()
    v = torch.stack((table[c & 15], table[c >> 4]), 2)
    s = scales[e].view(torch.float8_e4m3fn).float()
    return (v.view(*s.shape, 16) * s.unsqueeze(2)).view(v.shape[0], -1)


def _plan(ids, E):
    """Places in expert order: (slots in that order, offsets of the experts, the place of each slot)."""
    flat = ids.view(-1).long()
    real = (flat >= 0) & (flat < E)
    key = torch.where(real, flat, E)
    order = torch.sort(key, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    places = torch.empty_like(order)
    places[order] = torch.arange(order.numel(), device=order.device)
    rows = torch.where(real[order], order, -1)
    return rows.int(), offsets.int(), torch.where(real, places, -1).view(ids.shape).int()


def _gate(a, kind):
    if kind == "silu":
        return a * torch.sigmoid(a)
    return 0.5 * a * (1 + torch.tanh(0.7978845608028654 * (a + 0.044715 * a * a * a)))


def _plain(s):
    E, k = s["E"], s["k"]
    if s["op"] == "route":
        l = s["logits"].float()
        if s["b"] is None:
            key = l
        elif s["score"] == "softmax":
            key = torch.softmax(l.double(), 1) + s["b"].double()
        else:
            key = 1 / (1 + torch.exp(-l.double())) + s["b"].double()
        ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
        p = torch.softmax(l, 1) if s["score"] == "softmax" else 1 / (1 + torch.exp(-l))
        p = torch.gather(p, 1, ids)
        if s["normalize"]:
            p = p / p.sum(1, keepdim=True)
        return ids.int(), p * s["scale"]
    if s["op"] == "plan":
        return _plan(s["ids"], E)
    if s["op"] == "gemm":
        R, at = s["T"] * k, s["offsets"].tolist()
        out = torch.empty(R, s["N"], dtype=TYPES[s["out"]], device=s["x"].device)
        x = s["x"] if s["rows"] is None else s["x"][(s["rows"] // k).long()]
        for e in range(E):
            if at[e] < at[e + 1]:
                out[at[e]:at[e + 1]] = (x[at[e]:at[e + 1]].float() @ _weight(s["w"], e).t()) * s["w"][2][e]
        return out
    rows, offsets, _ = _plan(s["ids"], E)
    at = offsets.tolist()
    out = torch.zeros(s["x"].shape, device=s["x"].device)
    p = s["p"].view(-1)
    for e in range(E):
        if at[e] < at[e + 1]:
            slot = rows[at[e]:at[e + 1]].long()
            x = s["x"][slot // k].float()
            h = _gate((x @ _weight(s["gate"], e).t()) * s["gate"][2][e], s["act"])
            h = h * ((x @ _weight(s["up"], e).t()) * s["up"][2][e])
            y = (h @ _weight(s["down"], e).t()) * s["down"][2][e]
            out[slot // k] += y * p[slot].unsqueeze(1)  # (a token chooses an expert once)
    return out.to(s["x"].dtype)


def run(s):
    if not own:
        return _plain(s)
    import w4a16_nvfp4_dense_amd as ffn
    if s["op"] == "route":
        score = ffn.SCORE_SOFTMAX if s["score"] == "softmax" else ffn.SCORE_SIGMOID
        return ffn.moe_route(s["logits"], s["k"], score, bias=s["b"], normalize=s["normalize"], scale=s["scale"])
    if s["op"] == "plan":
        return ffn.moe_plan(s["ids"], s["E"])
    if s["op"] == "gemm":
        return ffn.moe_gemm(s["x"], s["offsets"], ffn.MoeDeviceWeight(*s["w"]), rows=s["rows"], top_k=s["k"] if s["gather"] else 1,
                            out_dtype=TYPES[s["out"]])
    act = ffn.ACT_SILU if s["act"] == "silu" else ffn.ACT_GELU_TANH
    return ffn.moe_forward(s["x"], s["ids"], s["p"], ffn.MoeDeviceWeight(*s["gate"]), ffn.MoeDeviceWeight(*s["up"]),
                           ffn.MoeDeviceWeight(*s["down"]), act)


def _experts_met(case):
    """How many experts have a row, on average over choices of k distinct experts a token, all as likely."""
    E = case["E"]
    return E * (1 - (1 - case["k"] / E) ** (case["T"] - case.get("pad", 0)))


def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        return {"bytes": T * E * SIZE[case["dtype"]] + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if case["op"] == "plan":
        return {"bytes": 12 * T * k + 4 * (E + 1), "flops": 2 * T * k}
    K, N, e = case["K"], case["N"], SIZE[case["dtype"]]
    met = _experts_met(case)
    if case["op"] == "gemm":
        moved = (T * K * e + 4 * T * k) if case["gather"] else T * k * K * e
        return {"bytes": int(met * (N * K * NVFP4_BYTES + 4) + moved + 4 * (E + 1) + T * k * N * SIZE[case["out"]]),
                "flops": 2 * T * k * K * N}
    real = T - case["pad"]
    return {"bytes": int(met * 3 * (N * K * NVFP4_BYTES + 4) + (real + T) * K * e + 8 * T * k),
            "flops": 6 * real * k * K * N}


# ---------------------------------------------------------------- the definitions, 64 bits


def _real(w, e):
    """Expert e's weight in 64 bits, from the fields of its codes and of its scales' bytes."""
    codes, scales, scale2 = w
    q = torch.stack((codes[e].bitwise_and(15), codes[e].bitwise_right_shift(4)), dim=-1).flatten(1).to(torch.int64)
    exponent, mantissa = q.bitwise_right_shift(1) & 3, q & 1
    v = torch.where(exponent == 0, 0.5 * mantissa.double(),
                    torch.ldexp(1 + 0.5 * mantissa.double(), (exponent - 1).double()))
    v = torch.where(q >= 8, -v, v)
    b = scales[e].to(torch.int64)
    exponent, mantissa = b.bitwise_right_shift(3) & 15, (b & 7).double()
    s = torch.where(exponent == 0, mantissa / 512, torch.ldexp(1 + mantissa / 8, (exponent - 7).double()))
    s = torch.where(b >= 128, -s, s)
    return v * s.repeat_interleave(16, dim=1) * scale2[e].double()


def exact(case, seed):
    s = prepare(case, seed)
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        l = s["logits"].double()
        if case["score"] == "softmax":
            z = torch.exp(l - torch.logsumexp(l, dim=1)[:, None])
        else:
            z = torch.special.expit(l)
        key = l if s["b"] is None else z + s["b"].double()
        best = torch.argsort(key.neg(), dim=1, stable=True).narrow(1, 0, k)
        v = z.take_along_dim(best, 1)
        if case["normalize"]:
            v = v / torch.linalg.vector_norm(v, ord=1, dim=1)[:, None]
        return best.to(torch.int32), v * case["scale"]
    if case["op"] == "plan":
        ids = s["ids"].flatten().cpu().tolist()
        members = [[] for _ in range(E)]
        for slot, e in enumerate(ids):
            if 0 <= e < E:
                members[e].append(slot)
        rows, offsets, places = [], [0], [-1] * len(ids)
        for slots in members:
            for slot in slots:
                places[slot] = len(rows)
                rows.append(slot)
            offsets.append(len(rows))
        rows += [-1] * (len(ids) - len(rows))
        return tuple(torch.tensor(v, dtype=torch.int32, device=DEV) for v in (rows, offsets)) + (
            torch.tensor(places, dtype=torch.int32, device=DEV).view(T, k),)
    if case["op"] == "gemm":
        out = torch.zeros(T * k, case["N"], dtype=torch.float64, device=DEV)
        edges = s["offsets"].cpu()
        for e in range(E):
            mine = torch.arange(int(edges[e]), int(edges[e + 1]), device=DEV)
            if mine.numel():
                token = mine if s["rows"] is None else torch.div(s["rows"][mine].long(), k, rounding_mode="floor")
                out.index_copy_(0, mine, torch.mm(s["x"][token].double(), _real(s["w"], e).t()))
        return out
    out = torch.zeros(T, case["K"], dtype=torch.float64, device=DEV)
    for e in range(E):
        token, choice = torch.nonzero(s["ids"] == e, as_tuple=True)
        if token.numel() == 0:
            continue
        x = s["x"].index_select(0, token).double()
        a, u = torch.mm(x, _real(s["gate"], e).t()), torch.mm(x, _real(s["up"], e).t())
        if case["act"] == "silu":
            h = a / (1.0 + torch.exp(-a)) * u
        else:
            h = torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a.pow(3))) * a * u
        out.index_add_(0, token, torch.mm(h, _real(s["down"], e).t()).mul_(s["p"][token, choice].double()[:, None]))
    return out
