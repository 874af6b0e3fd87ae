"""Int8 (W8A8) operators on the GPU against a plain numpy implementation in 64
bits (needs an MI355X).

What is exact and what is not:
  - the product's integer sums are exact, and its epilogue is a fixed chain of
    fp32 roundings, so the product is compared bit for bit with numpy: float64
    sums of integers (exact below 2^53), then the chain in float32;
  - the row quantiser is a fixed chain of fp32 roundings: bit for bit;
  - the norm's y has rounding error: the sum of squares of K <= 65536 terms is
    taken in at most 64 sequential additions per thread and 26 tree steps, so
    its relative error is below 100 * 2^-24 = 6e-6, half of that under the
    square root, and four more roundings: 3.3e-6, taken as 4e-6. A scale is
    then within 4e-6 of its value and a code within 127 * 2 * 4e-6 = 1.1e-3
    of one half from y / s;
  - h = act(g) u: g and u have three roundings each, e^z and 1 / (1 + e^z) are
    hardware approximations of 1 ulp with an argument error of |z| 2^-24 that
    a factor z e^-z <= 0.37 damps: below 2e-6 of the row's maximum, so a code
    is within 127 * 2 * 2e-6 = 5e-4, taken as 1e-3, of one half.
"""
import numpy as np
import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn

pytestmark = pytest.mark.gpu

F32 = np.float32
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def rounded(v, dtype):
    """A float32 array rounded once to dtype, as a torch tensor."""
    return torch.from_numpy(np.ascontiguousarray(v, dtype=F32)).to(TORCH[dtype])


def np_of(t):
    return t.detach().cpu().to(torch.float64 if t.dtype == torch.float64 else torch.float32).numpy()


def same_bits(a, b):
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(
        a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


def quant32(v):
    """The row rule in float32, step by step."""
    v = np.asarray(v, F32)
    amax = np.max(np.abs(v), axis=1)
    with np.errstate(all="ignore"):
        s = (amax / F32(127)).astype(F32)
        live = np.isfinite(amax) & (s >= np.finfo(F32).tiny)
        inv = np.where(live, F32(1) / np.where(live, s, F32(1)), F32(0)).astype(F32)
        q = np.where(live[:, None], np.rint((v * inv[:, None]).astype(F32)), 0)
    scale = np.where(live, s, np.where(np.isfinite(amax), F32(0), F32(np.nan))).astype(F32)
    return np.nan_to_num(q).astype(np.int8), scale


def product32(xq, xs, wq, ws, bias=None):
    sums = xq.astype(np.float64) @ wq.astype(np.float64).T
    y = (sums.astype(F32) * xs[:, None]).astype(F32) * ws[None, :]
    return y.astype(F32) if bias is None else (y.astype(F32) + bias[None, :]).astype(F32)


def make_tokens(rng, M, K):
    q = rng.integers(-128, 128, (M, K)).astype(np.int8)
    return q, rng.uniform(0.001, 0.02, M).astype(F32)


def make_weight(rng, N, K):
    q = rng.integers(-127, 128, (N, K)).astype(np.int8)
    return q, (rng.uniform(0.5, 2.0, N) / (127 * np.sqrt(K))).astype(F32)


def dev(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def weight_on(q, s):
    return ffn.Int8DeviceWeight(*dev(q, s))


# ------------------------------------------------------------------ quantiser


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 48), (3, 1040), (2, 5120), (7, 8208), (2, 17408), (1, 32768), (2, 65536)])
def test_quantize(rows, cols, dtype):
    rng = np.random.default_rng(rows * 100003 + cols)
    x = rounded(rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1))), dtype)
    q, s = quant32(np_of(x))
    codes, scales = ffn.int8_quantize(x.cuda())
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.array_equal(scales.cpu().numpy(), s)


def test_quantize_special_rows():
    """Zeros, magnitudes too small for a scale, the smallest that has one,
    the largest, ties, and rows with an infinity or a NaN, each beside an
    ordinary row that must not notice."""
    K = 64
    rng = np.random.default_rng(5)
    v = rng.standard_normal((9, K)).astype(F32)
    v[0] = 0.0
    v[1] = rng.uniform(-1, 1, K) * 1e-38
    v[2] = np.linspace(-1, 1, K) * F32(127) * np.finfo(F32).tiny * F32(1.001)
    v[3] *= F32(1e38) / np.abs(v[3]).max()
    v[4] = (np.arange(K) - 31.5)          # scale 32.5 / 127: no ties
    v[5] = np.where(np.arange(K) == 0, 127.0, np.arange(K) + 0.5)  # scale 1: ties to even
    v[6, 3] = np.inf
    v[7, 9] = np.nan
    v[7, 10] = -np.inf
    q, s = quant32(v)
    codes, scales = ffn.int8_quantize(torch.from_numpy(v).cuda())
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert s[0] == 0 and s[1] == 0 and s[2] > 0 and np.isnan(s[6]) and np.isnan(s[7]) and s[8] > 0
    assert not q[6].any() and not q[7].any() and list(q[5][:5]) == [127, 2, 2, 4, 4]


def test_quantize_weight_shape():
    """A weight of the decode shape (17408 x 5120), every element."""
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(17408, 5120, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    q = ffn.int8_quantize_weight(w)
    rows = [0, 1, 8191, 17407]
    qr, sr = quant32(np_of(w[rows]))
    assert np.array_equal(q.codes[rows].cpu().numpy(), qr) and np.array_equal(q.scales[rows].cpu().numpy(), sr)
    back = q.codes.float() * q.scales[:, None]
    assert bool(((back - w.float()).abs() <= q.scales[:, None] * 0.5001).all())


# ----------------------------------------------------------------------- norm


def norm64(x, r, w, eps, offset):
    t = np_of(x).astype(np.float64)
    if r is not None:
        t = t + np_of(r).astype(np.float64)
    y = t / np.sqrt(np.mean(t * t, axis=1, keepdims=True) + eps) * (offset + np_of(w).astype(np.float64))
    return t, y


def check_norm(codes, scales, y):
    s = np.max(np.abs(y), axis=1) / 127
    got_s = scales.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got_s - s) <= 4e-6 * s), np.max(np.abs(got_s / s - 1))
    far = np.abs(codes.cpu().numpy() - y / s[:, None])
    assert far.max() <= 0.5 + 1.1e-3, far.max()


@pytest.mark.parametrize("M,K,dtype,wdtype,residual,offset", [
    (1, 16, "bf16", "bf16", True, 0.0),
    (1, 5120, "bf16", "bf16", True, 0.0),
    (3, 5376, "bf16", "f32", True, 1.0),
    (2, 1040, "f16", "f16", False, 0.0),
    (5, 656, "f16", "bf16", True, 1.0),
    (4, 17408, "f32", "f32", True, 0.0),
    (2, 48, "f32", "f16", False, 1.0),
    (1, 65536, "bf16", "bf16", True, 0.0),
    (300, 2064, "bf16", "bf16", True, 0.0),
])
def test_rmsnorm(M, K, dtype, wdtype, residual, offset):
    rng = np.random.default_rng(M * 7919 + K)
    x = rounded(rng.standard_normal((M, K)), dtype)
    r = rounded(3 * rng.standard_normal((M, K)), dtype) if residual else None
    w = rounded(1 - offset + 0.2 * rng.standard_normal(K), wdtype)
    y_out = torch.empty((M, K), dtype=TORCH[dtype], device="cuda")
    codes, scales, total = ffn.int8_rmsnorm(x.cuda(), w.cuda(), 1e-6, residual=None if r is None else r.cuda(),
                                            weight_offset=offset, y_out=y_out)
    t, y = norm64(x, r, w, 1e-6, offset)
    check_norm(codes, scales, y)
    step = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[dtype]  # of one rounding
    assert np.all(np.abs(np_of(y_out) - y) <= np.abs(y) * (step + 4e-6) + 1e-7)
    if residual:
        # the sum is rounded to fp32, then to the type: numpy does the same
        assert same_bits(total, rounded((np_of(x) + np_of(r)).astype(F32), dtype))
    else:
        assert total is None
    # the same call again, in place of the residual, gives the same bits
    c2, s2, t2 = ffn.int8_rmsnorm(x.cuda(), w.cuda(), 1e-6, residual=None if r is None else r.cuda(), weight_offset=offset)
    assert same_bits(codes, c2) and same_bits(scales, s2)


@pytest.mark.parametrize("alias", ["x", "residual"])
def test_rmsnorm_in_place(alias):
    rng = np.random.default_rng(8)
    M, K = 37, 5120
    x, r = (rounded(rng.standard_normal((M, K)), "bf16").cuda() for _ in range(2))
    w = rounded(1 + 0.1 * rng.standard_normal(K), "bf16").cuda()
    c0, s0, t0 = ffn.int8_rmsnorm(x, w, residual=r)
    c1, s1, t1 = ffn.int8_rmsnorm(x, w, residual=r, sum_out=x if alias == "x" else r)
    assert t1 is (x if alias == "x" else r)
    assert same_bits(c0, c1) and same_bits(s0, s1) and same_bits(t0, t1)


def test_rmsnorm_special_rows():
    """A row of zeros has codes and scale 0 (eps carries the root); rows with
    an infinity or a NaN have scale NaN and codes 0; the others stand."""
    rng = np.random.default_rng(9)
    v = rng.standard_normal((5, 512)).astype(F32)
    v[1] = 0
    v[2, 17] = np.inf
    v[3, 200] = np.nan
    w = np.ones(512, F32)
    codes, scales, _ = ffn.int8_rmsnorm(*dev(v, w))
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    assert scales[1] == 0 and np.isnan(scales[2]) and np.isnan(scales[3])
    assert not codes[1:4].any()
    _, y = norm64(torch.from_numpy(v[[0, 4]]), None, torch.from_numpy(w), 1e-6, 0.0)
    check_norm(torch.from_numpy(codes[[0, 4]]), torch.from_numpy(scales[[0, 4]]), y)


# -------------------------------------------------------------------- product


@pytest.mark.parametrize("M,K,N,dtype,bias", [
    (1, 16, 1, "f32", False),
    (1, 256, 512, "bf16", False),
    (1, 5120, 333, "bf16", True),
    (2, 48, 17, "f32", True),
    (7, 1040, 100, "f16", True),
    (16, 272, 130, "f32", False),
    (17, 4112, 255, "bf16", False),
    (32, 512, 64, "f16", False),
    (33, 320, 96, "f32", True),
    (48, 1936, 51, "bf16", True),
    (64, 1024, 192, "f32", False),
    (65, 16, 5, "f32", True),
    (65, 128, 128, "bf16", False),
    (100, 144, 300, "f32", True),
    (128, 2048, 257, "f16", True),
    (129, 4112, 129, "f32", False),
    (256, 640, 512, "bf16", False),
    (300, 1168, 1027, "f32", True),
    (513, 256, 640, "bf16", True),
    (1025, 400, 260, "f32", False),
])
def test_gemm(M, K, N, dtype, bias):
    rng = np.random.default_rng(M * 31 + K * 7 + N)
    xq, xs = make_tokens(rng, M, K)
    wq, ws = make_weight(rng, N, K)
    b = rng.standard_normal(N).astype(F32) if bias else None
    out = ffn.int8_gemm(*dev(xq, xs), weight_on(wq, ws), bias=None if b is None else dev(b)[0], out_dtype=TORCH[dtype])
    assert same_bits(out, rounded(product32(xq, xs, wq, ws, b), dtype))


def test_gemm_largest_sums():
    """Codes of -128 and +-127 in one sign: the largest sums int32 has to hold,
    at the longest reduction."""
    M, K, N = 3, 65536, 33
    xq = np.full((M, K), -128, np.int8)
    xq[1] = 127
    wq = np.full((N, K), -128, np.int8)
    wq[5] = 127
    xs, ws = np.ones(M, F32), np.ones(N, F32)
    out = ffn.int8_gemm(*dev(xq, xs), weight_on(wq, ws), out_dtype=torch.float32)
    assert same_bits(out, rounded(product32(xq, xs, wq, ws), "f32"))


@pytest.mark.parametrize("M", [1, 16, 40, 64, 65, 200])
def test_gemm_nan_scale_stays_in_its_row(M):
    rng = np.random.default_rng(M)
    K, N = 512, 96
    xq, xs = make_tokens(rng, M, K)
    wq, ws = make_weight(rng, N, K)
    ref = product32(xq, xs, wq, ws)
    xs[M // 2] = np.nan
    out = ffn.int8_gemm(*dev(xq, xs), weight_on(wq, ws), out_dtype=torch.float32).cpu().numpy()
    assert np.isnan(out[M // 2]).all()
    keep = np.arange(M) != M // 2
    assert np.array_equal(out[keep], ref[keep])


@pytest.mark.parametrize("M,K,N,dtype,bias", [
    (1024, 272, 10250, "f32", True),    # 256 x 256 tiles, fewer than compute units, a short last stage
    (1792, 144, 19001, "bf16", False),  # two rounds of them and a shared rest, ragged channels
    (2300, 128, 20480, "f16", True),    # one stage a tile, ragged tokens
    (250, 400, 16500, "f32", False),    # 256 x 128 tiles
    (256, 2064, 17408, "bf16", True),
    (1, 5120, 30000, "f32", True),      # weights read non-temporally
    (40, 4112, 33333, "bf16", False),
    (64, 8208, 16500, "f32", False),
    (37, 2064, 5000, "f32", True),      # 64 x 64 tiles
    (700, 1040, 3000, "f16", False),
])
def test_gemm_large(M, K, N, dtype, bias):
    """Every tile shape at sizes with several rounds of tiles, shared tiles and
    ragged ends, bit for bit: integer sums in float64 on the GPU are exact, and
    torch's fp32 products and sums round as the chain does."""
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(M, generator=g, device="cuda") / 64
    ws = torch.rand(N, generator=g, device="cuda") / 64
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    ref = (xq.double() @ wq.double().t().contiguous()).float() * xs[:, None] * ws
    if bias:
        ref = ref + b
    workspace = torch.full((max(16, ffn.int8_gemm_workspace_bytes(M, K, N)),), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(2):  # the second call finds what the first one left
        out = ffn.int8_gemm(xq, xs, ffn.Int8DeviceWeight(wq, ws), bias=b, out_dtype=TORCH[dtype], workspace=workspace)
        assert same_bits(out, ref.to(TORCH[dtype]))


@pytest.mark.parametrize("M,K,N,act", [(1024, 144, 5136, 0), (1300, 256, 10240, 1), (250, 272, 8256, 0), (500, 528, 1040, 1)])
def test_dual_large(M, K, N, act):
    """The gated product on the tile shapes of many tokens: the same bits as on
    those of few (which the tests below hold against 64 bits)."""
    xq, xs, gate, up, down = _config(M, K, N, M + N)
    hq, hs = ffn.int8_dual_gemm(xq, xs, gate, up, act)
    for lo in range(0, M, 61):
        q, s = ffn.int8_dual_gemm(xq[lo:lo + 3], xs[lo:lo + 3], gate, up, act)
        assert same_bits(q, hq[lo:lo + 3]) and same_bits(s, hs[lo:lo + 3])
    out = ffn.int8_forward(xq, xs, gate, up, down, act)
    assert same_bits(out, ffn.int8_gemm(hq, hs, down))


@pytest.mark.parametrize("K,N", [(5120, 17408), (17408, 5120), (1040, 531)])
def test_gemm_rows_do_not_depend_on_the_batch(K, N):
    """Row m of every batch has the bits of a call on that row alone."""
    g = torch.Generator(device="cuda").manual_seed(K)
    M = 640
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(M, generator=g, device="cuda") + 0.5
    w = ffn.Int8DeviceWeight(torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8),
                             torch.rand(N, generator=g, device="cuda") + 0.5)
    whole = ffn.int8_gemm(xq, xs, w)
    for lo, m in ((0, 1), (3, 2), (5, 13), (20, 17), (40, 48), (100, 64), (170, 65), (240, 128), (300, 300)):
        part = ffn.int8_gemm(xq[lo:lo + m], xs[lo:lo + m], w)
        assert same_bits(part, whole[lo:lo + m]), (lo, m)


def test_gemm_outputs_do_not_pass_the_end():
    """Ragged channels and tokens leave what lies behind the output alone."""
    rng = np.random.default_rng(2)
    for M, K, N in ((1, 64, 7), (20, 64, 33), (70, 192, 131), (260, 192, 259)):
        xq, xs = make_tokens(rng, M, K)
        wq, ws = make_weight(rng, N, K)
        buf = torch.full((M * N + 4096,), 7.0, device="cuda")
        ffn.int8_gemm(*dev(xq, xs), weight_on(wq, ws), out=buf[:M * N].view(M, N))
        assert bool((buf[M * N:] == 7.0).all())
        assert same_bits(buf[:M * N].view(M, N), rounded(product32(xq, xs, wq, ws), "f32"))


# -------------------------------------------------------------- gated products


def act64(g, act):
    if act == ffn.ACT_SILU:
        return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


GATED = [
    (1, 16, 16, 0), (1, 256, 512, 0), (3, 1040, 96, 1), (9, 512, 272, 0), (16, 656, 160, 1), (17, 256, 336, 1),
    (32, 512, 512, 0), (50, 272, 144, 0), (64, 1024, 80, 1), (65, 400, 208, 0), (130, 640, 528, 1), (300, 256, 304, 0),
]


@pytest.mark.parametrize("M,K,N,act", GATED)
def test_dual_and_forward(M, K, N, act):
    rng = np.random.default_rng(M * 17 + K + N)
    xq, xs = make_tokens(rng, M, K)
    gq, gs = make_weight(rng, N, K)
    uq, us = make_weight(rng, N, K)
    dq, ds = make_weight(rng, K, N)
    x = dev(xq, xs)
    gate, up, down = weight_on(gq, gs), weight_on(uq, us), weight_on(dq, ds)
    hq, hs = ffn.int8_dual_gemm(*x, gate, up, act)

    def real(q, s):
        return q.astype(np.float64) * s.astype(np.float64)[:, None]

    h = act64(real(xq, xs) @ real(gq, gs).T, act) * (real(xq, xs) @ real(uq, us).T)
    s = np.abs(h).max(axis=1) / 127
    got_q, got_s = hq.cpu().numpy(), hs.cpu().numpy()
    assert np.all(np.abs(got_s - s) <= 4e-6 * s)
    assert np.abs(got_q - h / s[:, None]).max() <= 0.5 + 1e-3
    # the down projection of these codes, bit for bit, and the whole forward
    ref = product32(got_q, got_s, dq, ds)
    for dtype in ("bf16", "f16", "f32"):
        out = ffn.int8_forward(*x, gate, up, down, act, out_dtype=TORCH[dtype])
        assert same_bits(out, rounded(ref, dtype)), dtype


def _config(M, K, N, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(r, c):
        return (torch.randn(r, c, generator=g, device="cuda") * 32).round().clamp(-127, 127).to(torch.int8)

    def weight(r, c):
        return ffn.Int8DeviceWeight(codes(r, c), (torch.rand(r, generator=g, device="cuda") + 0.5) / (32 * c ** 0.5))

    return codes(M, K), torch.rand(M, generator=g, device="cuda") / 32, weight(N, K), weight(N, K), weight(K, N)


@pytest.mark.parametrize("K,N,act", [(5120, 17408, 0), (5376, 21504, 1)])
def test_forward_rows_do_not_depend_on_the_batch(K, N, act):
    """The decode shapes: every batch size's rows have the bits of the M = 1 call."""
    xq, xs, gate, up, down = _config(200, K, N, K)
    one = torch.cat([ffn.int8_forward(xq[m:m + 1], xs[m:m + 1], gate, up, down, act) for m in range(0, 200, 9)])
    for M in (2, 8, 16, 17, 32, 40, 64, 65, 128, 200):
        out = ffn.int8_forward(xq[:M], xs[:M], gate, up, down, act)
        n = (M + 8) // 9
        assert same_bits(out[0:M:9], one[:n]), M


@pytest.mark.parametrize("K,N", [(16, 16), (256, 512), (272, 1040), (512, 24560), (512, 24576), (512, 24592),
                                 (5120, 17408), (8192, 16384), (20480, 1024)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_forward_of_one_token_is_its_parts(K, N, out_dtype):
    """One token's h is quantised inside the down product where it is short enough: the bits are those of the
    two calls, whose quantisation is a launch of its own."""
    xq, xs, gate, up, down = _config(2, K, N, 11)
    for act in (ffn.ACT_SILU, ffn.ACT_GELU_TANH):
        hq, hs = ffn.int8_dual_gemm(xq[:1], xs[:1], gate, up, act)
        ref = ffn.int8_gemm(hq, hs, down, out_dtype=out_dtype)
        assert same_bits(ffn.int8_forward(xq[:1], xs[:1], gate, up, down, act, out_dtype), ref)
    # nothing but zeros, and a NaN
    zero = ffn.int8_forward(torch.zeros_like(xq[:1]), xs[:1], gate, up, down, out_dtype=out_dtype)
    assert bool((zero == 0).all())
    nan = ffn.int8_forward(xq[:1], torch.full_like(xs[:1], float("nan")), gate, up, down, out_dtype=out_dtype)
    assert bool(nan.isnan().all())


def test_forward_decode_shape_against_64_bits():
    M, K, N = 4, 5120, 17408
    xq, xs, gate, up, down = _config(M, K, N, 1)
    hq, hs = ffn.int8_dual_gemm(xq, xs, gate, up)

    def real(w):
        return w.codes.double() * w.scales.double()[:, None]

    x = xq.double() * xs.double()[:, None]
    g, u = x @ real(gate).t().contiguous(), x @ real(up).t().contiguous()
    h = g / (1 + torch.exp(-g)) * u
    s = h.abs().amax(1) / 127
    assert bool(((hs.double() - s).abs() <= 4e-6 * s).all())
    assert float((hq.double() - h / s[:, None]).abs().max()) <= 0.5 + 1e-3
    out = ffn.int8_forward(xq, xs, gate, up, down, out_dtype=torch.float32)
    # integer sums in float64 are exact (a sum of real values would leave noise
    # where the integers cancel to zero)
    sums = hq.double() @ down.codes.double().t().contiguous()
    ref = sums * hs.double()[:, None] * down.scales.double()
    # three fp32 roundings of each value
    assert bool(((out.double() - ref).abs() <= 2e-7 * ref.abs() + 1e-30).all())


def test_forward_nan_row():
    """A token with a NaN (scale NaN, codes 0) gives a NaN row; the others stand."""
    xq, xs, gate, up, down = _config(70, 512, 1024, 4)
    for M in (5, 70):
        ref = ffn.int8_forward(xq[:M], xs[:M], gate, up, down)
        q, s = xq[:M].clone(), xs[:M].clone()
        q[2], s[2] = 0, float("nan")
        out = ffn.int8_forward(q, s, gate, up, down)
        assert bool(out[2].isnan().all())
        keep = [m for m in range(M) if m != 2]
        assert same_bits(out[keep], ref[keep])


def test_zero_tokens_and_zero_rows():
    xq, xs, gate, up, down = _config(3, 256, 512, 6)
    assert ffn.int8_forward(xq[:0], xs[:0], gate, up, down).shape == (0, 256)
    assert ffn.int8_gemm(xq[:0], xs[:0], gate).shape == (0, 512)
    c, s = ffn.int8_quantize(torch.empty(0, 64, device="cuda"))
    assert c.shape == (0, 64) and s.shape == (0,)
    z = torch.zeros_like(xq)
    assert not bool(ffn.int8_forward(z, xs, gate, up, down).any())


# ------------------------------------------------- from the framework's weights


def test_prepare_weight():
    """NVFP4 -> int8: every code and scale of the dequantised rows, a row of
    zeros, a NaN scale byte, a negative scale2."""
    import ffn_inputs as fi
    case = fi.make_small(1, 1056, 96, seed=21)
    w = case.gate
    scales = w.scales.copy()
    codes = w.codes.copy()
    codes[3] = 0
    scales[7, 2] = 0x7F
    e2m1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], F32)
    sc = torch.from_numpy(scales).view(torch.float8_e4m3fn).float().numpy()
    vals = np.empty((96, 1056), F32)
    vals[:, 0::2], vals[:, 1::2] = e2m1[codes & 15], e2m1[codes >> 4]
    vals *= np.repeat(sc, 16, axis=1)
    for scale2 in (1.0, -0.0625, 0.3):
        d = ffn.DeviceWeight(*dev(codes, scales), scale2)
        got = ffn.int8_prepare_weight(d)
        q, s = quant32(vals)
        assert np.array_equal(got.codes.cpu().numpy(), q)
        assert np.array_equal(got.scales.cpu().numpy(), (s * F32(scale2)).astype(F32), equal_nan=True)
        assert s[3] == 0 and np.isnan(s[7])


def test_block_from_nvfp4_weights():
    """norm -> FFN -> residual over weights prepared from NVFP4 against the
    same layer in 64 bits on the NVFP4 weights. What separates them is the
    8-bit rounding, whose relative error is a row's maximum over its rms,
    divided by 127 sqrt(12): about 3.5 for x (0.8%), 5 for the weights (1.1%)
    and up to 15 for a product of normals, h (3.4%). In quadrature, with g and
    u each carrying x's and a weight's: 4.1%, held to twice that."""
    import ffn_inputs as fi
    import oracle
    case = fi.make_small(8, 1024, 2048, seed=22)
    rng = np.random.default_rng(22)
    x, r = (rounded(rng.standard_normal((8, 1024)), "bf16") for _ in range(2))
    w = rounded(1 + 0.1 * rng.standard_normal(1024), "bf16")
    gate, up, down = (ffn.int8_prepare_weight(ffn.DeviceWeight.from_host(v)) for v in (case.gate, case.up, case.down))
    codes, scales, total = ffn.int8_rmsnorm(x.cuda(), w.cuda(), residual=r.cuda())
    out = ffn.int8_forward(codes, scales, gate, up, down, case.act)
    _, y = norm64(x, r, w, 1e-6, 0.0)
    case.x_bits[:] = torch.from_numpy(y).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    ref = oracle.ffn(case)
    err = np.linalg.norm(np_of(out) - ref) / np.linalg.norm(ref)
    assert err < 0.082, err


# ----------------------------------------------------------- streams and graphs


def test_other_stream_and_caller_buffers():
    xq, xs, gate, up, down = _config(33, 1024, 2048, 7)
    ref = ffn.int8_forward(xq, xs, gate, up, down)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [ffn.int8_forward(xq, xs, gate, up, down, stream=side) for _ in range(4)]
    ws = torch.full((ffn.int8_workspace_bytes(33, 1024, 2048),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(ref, float("nan"))
    ffn.int8_forward(xq, xs, gate, up, down, out=out, workspace=ws)
    side.synchronize()
    torch.cuda.synchronize()
    for o in outs + [out]:
        assert same_bits(o, ref)


@pytest.mark.parametrize("M", [1, 32, 300])
def test_two_streams_at_once(M):
    """Forwards on two streams, each with its own workspace, beside each other on the card: shared tiles of both
    are finished right."""
    K, N = 5120, 17408
    xq, xs, gate, up, down = _config(M, K, N, 21)
    ref = ffn.int8_forward(xq, xs, gate, up, down)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [torch.empty(ffn.int8_workspace_bytes(M, K, N), dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [[torch.empty_like(ref) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, ws, out in zip(streams, spaces, outs):
            ffn.int8_forward(xq, xs, gate, up, down, out=out[i], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for out in outs:
        for o in out:
            assert same_bits(o, ref)


@pytest.mark.parametrize("M", [1, 24, 80, 300])
def test_graph_replays(M):
    """Captured norm, forward and product: every replay against the eager
    result, with other work and other inputs between the replays."""
    K, N = 1024, 2048
    xq, xs, gate, up, down = _config(M, K, N, 11)
    x = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    r = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(K, device="cuda", dtype=torch.bfloat16)
    codes, scales, total = ffn.int8_rmsnorm(x, w, residual=r)
    ws = torch.empty(max(1, ffn.int8_workspace_bytes(M, K, N)), dtype=torch.uint8, device="cuda")
    gws = torch.empty(max(1, ffn.int8_gemm_workspace_bytes(M, K, N)), dtype=torch.uint8, device="cuda")
    out = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
    prod = torch.empty(M, N, device="cuda", dtype=torch.float32)

    def step(stream=None):
        ffn.int8_rmsnorm(x, w, residual=r, codes=codes, scales=scales, sum_out=total, stream=stream)
        ffn.int8_forward(codes, scales, gate, up, down, out=out, workspace=ws, stream=stream)
        ffn.int8_gemm(codes, scales, gate, out=prod, workspace=gws, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for k in range(4):
        x.copy_(torch.randn(M, K, device="cuda"))
        step()
        torch.cuda.synchronize()
        ref = [t.clone() for t in (codes, scales, total, out, prod)]
        for t in (codes, scales, total, out, prod):
            t.zero_()
        ws.fill_(k)
        gws.fill_(255 - k)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((codes, scales, total, out, prod), ref):
            assert same_bits(a, b), k


# ----------------------------------------------------------- beyond 32 bits
def test_weight_past_4_gib():
    """65600 x 65536 codes: the channels at either end, exactly (sums of at most 65536 * 2^14 = 2^30)."""
    K, N = 65536, 65600
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=g, device="cuda") / K
    for M in (1, 3, 40):
        xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
        xs = torch.rand(M, generator=g, device="cuda")
        out = ffn.int8_gemm(xq, xs, ffn.Int8DeviceWeight(w, ws), out_dtype=torch.float32)
        for at in (slice(0, 64), slice(N - 64, N)):
            sums = xq.double() @ w[at].double().t().contiguous()
            assert same_bits(out[:, at].contiguous(), sums.float() * xs[:, None] * ws[None, at]), (M, at)


def test_output_past_4_gib():
    M, K, N = 65536, 32, 65600
    g = torch.Generator(device="cuda").manual_seed(6)
    w = ffn.Int8DeviceWeight(torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8),
                             torch.rand(N, generator=g, device="cuda"))
    xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand(M, generator=g, device="cuda")
    out = ffn.int8_gemm(xq, xs, w)
    for m in (0, 32767, 32768, M - 1):
        assert same_bits(out[m:m + 1], ffn.int8_gemm(xq[m:m + 1], xs[m:m + 1], w)), m


def test_rows_past_4_gib():
    rows, cols = 65600, 65536
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    codes, scales = ffn.int8_quantize(x)
    for r in (0, 32767, 32768, rows - 1):
        q, s = ffn.int8_quantize(x[r:r + 1].clone())
        assert same_bits(codes[r:r + 1], q) and same_bits(scales[r:r + 1], s), r
