"""The sparse FFN's definitions in 64 bits, and bounds on what the kernels' roundings can add, for its tests.

The weights' values come from torch's float8 decoder and a table of the E2M1 values; nothing here is shared with the
library. U = 2^-24 is half a step of fp32, half = eps / 2 half a step of a 16-bit type, both relative."""
import math

import torch

import w4a16_nvfp4_dense_amd as ffn

DEV = "cuda"
U = 2.0 ** -24
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def half(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def experts(E, rows, cols, seed):
    """Random NVFP4 experts: every code, scales of both signs over 2^-3 .. 2^1, values of about cols ** -0.5."""
    g = gen(seed)
    codes = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(0x20, 0x48, (E, rows, cols // 16), generator=g, device=DEV, dtype=torch.uint8)
    sign = torch.randint(0, 2, scales.shape, generator=g, device=DEV, dtype=torch.uint8) << 7
    scale2 = (0.5 + torch.rand(E, generator=g, device=DEV)) / (2 * cols ** 0.5)
    return ffn.MoeDeviceWeight(codes, scales | sign, scale2)


def dense(w, e):
    """Expert e's weight in float64, scale2 included."""
    table = torch.tensor([*E2M1, *(-v for v in E2M1)], dtype=torch.float64, device=w.codes.device)
    c = w.codes[e].long()
    v = torch.stack((table[c & 15], table[c >> 4]), -1).flatten(1)
    return v * w.scales[e].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * w.scale2[e].double()


def product(x, w, e):
    """(W_e x, the bound of its error in fp32): K products, added in any order, and scale2."""
    d = dense(w, e)
    a = x.double()
    return a @ d.t(), (x.shape[1] + 2) * U * (a.abs() @ d.abs().t())


def gemm(x, offsets, w, rows=None, top_k=1):
    """(values, bound of the fp32 result's error) [R, N]; nan where no expert's rows are."""
    R = x.shape[0] if rows is None else rows.numel()
    src = x if rows is None else x[(rows // top_k).clamp(0, x.shape[0] - 1).long()]
    y = torch.full((R, w.rows), math.nan, dtype=torch.float64, device=x.device)
    b = torch.zeros_like(y)
    at = offsets.tolist()
    for e in range(w.experts):
        if at[e] < at[e + 1]:
            y[at[e]:at[e + 1]], b[at[e]:at[e + 1]] = product(src[at[e]:at[e + 1]], w, e)
    return y, b


def act_of(g, act):
    if act == ffn.ACT_SILU:
        return g * torch.sigmoid(g)
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))


def act_bound(g, act):
    """Relative error of g / (1 + e^z) in fp32: z to 4 U |z| (its products), the exponential's argument z log2(e) to
    another U |z|, so e^z to 6 U |z| + 2 U, a reciprocal to 2 U, a product and a sum: under 8 U (|z| + 1)."""
    z = g.abs() if act == ffn.ACT_SILU else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3).abs()
    return 8 * U * (z.clamp(max=200.0) + 1)


def forward(x, ids, weights, gate, up, down, act):
    """(out, bound of its error in x's type). Both gates have a slope below 1.13."""
    t = x.dtype
    T, k = ids.shape
    out = torch.zeros(T, x.shape[1], dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    size = torch.zeros_like(out)
    for e in range(gate.experts):
        tok, j = torch.nonzero(ids == e, as_tuple=True)
        if not tok.numel():
            continue
        g, gb = product(x[tok], gate, e)
        u, ub = product(x[tok], up, e)
        a = act_of(g, act)
        h = a * u
        hb = 1.13 * gb * (u.abs() + ub) + a.abs() * ub + act_bound(g, act) * h.abs() + 2 * U * h.abs()
        hb = hb + half(t) * (h.abs() + hb) + torch.finfo(t).tiny  # h's rounding, the only one to 16 bits before the result's
        d = dense(down, e)
        y = h @ d.t()
        yb = hb @ d.abs().t() + (h.shape[1] + 2) * U * ((h.abs() + hb) @ d.abs().t())
        p = weights[tok, j].double()[:, None]
        out.index_add_(0, tok, p * y)
        bound.index_add_(0, tok, p.abs() * yb)
        size.index_add_(0, tok, p.abs() * (y.abs() + yb))
    bound += 2 * (k + 1) * U * size
    return out, bound + half(t) * (out.abs() + bound) + torch.finfo(t).tiny


def within(got, ref, bound):
    """Whether every element is within its bound; says which is furthest."""
    got = got.double()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    worst = (err / bound.clamp_min(1e-300)).max().item() if err.numel() else 0.0
    assert worst <= 1, f"error {worst} times its bound"
    return True
