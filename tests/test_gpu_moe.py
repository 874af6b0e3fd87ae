"""GPU tests of the sparse FFN's operators against their definitions in 64 bits (moe_ref.py), with bounds made of the
roundings that the kernels' comments name."""
import math

import pytest
import torch

import moe_ref as ref
import w4a16_nvfp4_dense_amd as ffn
from moe_ref import DEV, U, gen, half

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ the choice


def route_ref(logits, k, score, bias, normalize, scale):
    """(ids, weights) in 64 bits; the same where fewer than k are available."""
    l = logits.double()
    s = torch.softmax(l, 1) if score == ffn.SCORE_SOFTMAX else torch.sigmoid(l)
    key = l.clone() if bias is None else s + bias.double()
    key[l == -math.inf] = -math.inf
    key = key + 0.0
    rank = torch.where(torch.isnan(key), torch.full_like(key, -1e308), key)
    order = torch.sort(rank, dim=1, descending=True, stable=True)
    ids, none = order.indices[:, :k], order.values[:, :k] == -math.inf
    w = torch.where(none, torch.zeros((), dtype=torch.float64, device=l.device), s.gather(1, ids))
    if normalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, torch.zeros_like(w), w / total)
    return torch.where(none, -1, ids).int(), w * scale


def check_route(logits, k, score, bias=None, normalize=True, scale=1.0):
    ids, w = ffn.moe_route(logits, k, score, bias=bias, normalize=normalize, scale=scale)
    rid, rw = route_ref(logits, k, score, bias, normalize, scale)
    assert torch.equal(ids, rid)
    # fp32: exp and the argument's subtraction ((|l| + 4) U), a tree sum of E terms, two divisions, two products, k terms
    l = logits.float().abs()
    l = torch.where(torch.isfinite(l), l, torch.zeros_like(l)).amax(1, keepdim=True).double()
    tol = (2 * l + 4 + math.ceil(math.log2(logits.shape[1])) + logits.shape[1] / 64 + k + 8) * U * 2
    nan = torch.isnan(rw)
    assert torch.equal(torch.isnan(w), nan)
    err = ((w.double() - rw).abs() - tol * rw.abs())[~nan]
    assert err.numel() == 0 or err.max() <= 1e-37
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 2, 2), (5, 63, 32), (7, 65, 6), (333, 160, 6), (2, 256, 1),
                                   (64, 257, 9), (9, 1024, 32), (1000, 8, 8), (4096, 128, 4)])
@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("score", [ffn.SCORE_SOFTMAX, ffn.SCORE_SIGMOID])
def test_route(T, E, k, dtype, score):
    g = gen(T * 31 + E)
    logits = (2 * torch.randn(T, E, generator=g, device=DEV)).to(dtype)
    bias = 0.2 * torch.randn(E, generator=g, device=DEV)
    check_route(logits, k, score)
    check_route(logits, k, score, normalize=False, scale=2.5)
    check_route(logits, k, score, bias=bias)
    check_route(logits, k, score, bias=torch.zeros_like(bias), normalize=False)


@pytest.mark.parametrize("bias", [None, 0.0])
@pytest.mark.parametrize("E", [5, 64, 200, 700])
def test_route_ties_go_to_the_lower_expert(E, bias):
    """Few values, so that nearly every choice is a tie; zeros of both signs are one value."""
    logits = torch.randint(-1, 2, (257, E), generator=gen(E), device=DEV).float()
    logits[::2] *= -1  # zeros of the other sign
    b = None if bias is None else torch.zeros(E, device=DEV)
    for score in (ffn.SCORE_SOFTMAX, ffn.SCORE_SIGMOID):
        check_route(logits, min(E, 8), score, bias=b)
    assert torch.equal(ffn.moe_route(torch.zeros(3, E, device=DEV), 4)[0],
                       torch.arange(4, device=DEV, dtype=torch.int32).expand(3, 4))


@pytest.mark.parametrize("score", [ffn.SCORE_SOFTMAX, ffn.SCORE_SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_masks_and_special_values(score, with_bias):
    E, k = 70, 5
    logits = torch.randn(8, E, generator=gen(1), device=DEV)
    logits[1] = -math.inf                # nothing is available
    logits[2] = -math.inf
    logits[2, [3, 69]] = torch.tensor([0.5, 0.25], device=DEV)  # two of five
    logits[3, ::2] = -math.inf
    logits[4] = torch.finfo(F).min       # the lowest value is still a value
    logits[5, 7] = math.nan
    logits[6] = math.nan
    logits[7, 69] = torch.finfo(F).max
    bias = torch.linspace(0, 1e-3, E, device=DEV) if with_bias else None
    ids, w = check_route(logits, k, score, bias=bias)
    assert (ids[1] == -1).all() and (w[1] == 0).all()
    assert set(ids[2].tolist()) == {3, 69, -1} and (w[2, 2:] == 0).all()
    assert (ids[6] >= 0).all() and torch.isnan(w[6]).all()
    if with_bias:  # an expert taken out by its bias
        bias[ids[0, 0].long()] = -math.inf
        again, _ = check_route(logits, k, score, bias=bias)
        assert ids[0, 0] not in again[0]


def test_route_close_keys_with_bias():
    """Scores a few units of fp32 apart, which 32 bits would put in another order."""
    E = 256
    logits = 1 + torch.arange(E, device=DEV).flip(0).float() * 2.0 ** -23
    bias = torch.rand(E, generator=gen(3), device=DEV) * 2.0 ** -24
    check_route(logits.expand(4, E).contiguous(), 8, ffn.SCORE_SIGMOID, bias=bias)


# -------------------------------------------------------------------- the plan


def plan_ref(ids, E):
    flat = ids.flatten().tolist()
    order = sorted((s for s in range(len(flat)) if 0 <= flat[s] < E), key=lambda s: (flat[s], s))
    rows = order + [-1] * (len(flat) - len(order))
    counts = [0] * E
    places = [-1] * len(flat)
    for i, s in enumerate(order):
        counts[flat[s]] += 1
        places[s] = i
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    return rows, offsets, places


def check_plan(ids, E):
    got = ffn.moe_plan(ids, E)
    for a, b in zip(got, plan_ref(ids, E)):
        assert a.flatten().tolist() == b
    return got


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (1, 1, 1024), (3, 32, 1024), (33, 2, 7), (63, 1, 2), (64, 1, 3),
                                   (65, 1, 3), (1024, 8, 128), (1025, 8, 128), (2048, 4, 1024), (8193, 1, 5),
                                   (12288, 1, 1), (16384, 8, 256), (20001, 3, 255)])
def test_plan(T, k, E):
    ids = torch.randint(0, E, (T, k), generator=gen(T + E), device=DEV, dtype=torch.int32)
    check_plan(ids, E)
    ids[torch.rand(T, k, generator=gen(5), device=DEV) < 0.3] = -1
    ids[-1, -1] = E            # just past the last expert
    ids[0, 0] = 2 ** 31 - 1
    check_plan(ids, E)


def test_plan_extremes():
    check_plan(torch.full((50, 3), -1, device=DEV, dtype=torch.int32), 9)   # nobody
    check_plan(torch.full((5000, 3), 8, device=DEV, dtype=torch.int32), 9)  # everybody with one expert
    check_plan(torch.full((7, 3), -(2 ** 31), device=DEV, dtype=torch.int32), 9)
    rows, offsets, places = ffn.moe_plan(torch.empty(0, 4, device=DEV, dtype=torch.int32), 6)
    assert rows.numel() == places.numel() == 0 and offsets.tolist() == [0] * 7


# ----------------------------------------------------------------- the product


def by_counts(counts):
    return torch.tensor([0, *counts], device=DEV, dtype=torch.int32).cumsum(0).int()


def check_gemm(x, offsets, w, rows=None, top_k=1, out_dtype=None):
    y, b = ref.gemm(x, offsets, w, rows, top_k)
    t = out_dtype or x.dtype
    R = y.shape[0]
    out = torch.full((R, w.rows), -77.0, dtype=t, device=DEV)
    ffn.moe_gemm(x, offsets, w, rows=rows, top_k=top_k, out_dtype=out_dtype, out=out)
    a, z = int(offsets[0]), int(offsets[-1])
    if t != F:
        b = b + half(t) * (y.abs() + b) + torch.finfo(t).tiny
    ref.within(out[a:z], y[a:z], b[a:z])
    assert (out[:a] == -77).all() and (out[z:] == -77).all()
    assert torch.equal(out, ffn.moe_gemm(x, offsets, w, rows=rows, top_k=top_k, out=out.clone()))
    return out


COUNTS = [[1], [0, 1, 0], [5, 0, 3], [16, 17, 15, 1], [31, 32, 33], [63, 64, 65, 0], [0, 0, 129, 127, 128], [300, 1],
          [2] * 40, [7, 90, 0, 0, 200, 33]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "_".join(map(str, c[:6])))
@pytest.mark.parametrize("K,N", [(32, 1), (64, 33), (96, 257), (160, 128), (256, 64), (672, 300)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gemm(counts, K, N, dtype):
    R = sum(counts)
    w = ref.experts(len(counts), N, K, R + K)
    x = torch.randn(R, K, generator=gen(R), device=DEV).to(dtype)
    check_gemm(x, by_counts(counts), w, out_dtype=F if N % 2 else None)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("K,N", [(2048, 5120), (5120, 96), (17408, 40), (4128, 1999)])
def test_gemm_long_reductions(K, N, dtype):
    counts = [1, 9, 0, 40]
    w = ref.experts(4, N, K, K)
    x = torch.randn(50, K, generator=gen(K), device=DEV).to(dtype)
    check_gemm(x, by_counts(counts), w)
    check_gemm(x, by_counts(counts), w, out_dtype=F)
    check_gemm(x[:1].contiguous(), by_counts([0, 1, 0, 0]), w)


@pytest.mark.parametrize("T,k,E", [(1, 4, 8), (40, 3, 5), (200, 6, 3), (700, 2, 4)])
def test_gemm_reads_rows_where_they_are(T, k, E):
    ids = torch.randint(0, E, (T, k), generator=gen(T), device=DEV, dtype=torch.int32)
    rows, offsets, _ = ffn.moe_plan(ids, E)
    w = ref.experts(E, 160, 192, 3)
    x = torch.randn(T, 192, generator=gen(4), device=DEV).to(BF)
    a = check_gemm(x, offsets, w, rows=rows, top_k=k)
    b = check_gemm(x[(rows // k).long()].contiguous(), offsets, w)
    assert torch.equal(a, b)


# Shapes that reach each of the kernels' variants: the stream of few rows, one tile of many experts' rows after
# another; tiles of 32, 64 and 128 rows, where there are enough of them for the device and where there are not.
VARIANTS = [
    ([40] + [0] * 9, 64, 700), ([100, 1, 0, 17] + [0] * 20, 160, 96), ([512] + [0] * 40, 256, 48),
    ([20, 31, 1, 17, 18], 672, 3000), ([40, 64, 31, 50], 160, 16500), ([25, 96, 33, 64], 288, 16384),
    ([200, 129, 33, 300], 96, 8192), ([70, 128, 1, 97], 160, 16501), ([64, 65, 129, 257], 672, 9000),
    ([70, 128, 1, 97], 224, 130), ([1000], 416, 700), ([90] * 40, 128, 513),
]


@pytest.mark.parametrize("counts,K,N", VARIANTS, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("wide", [False, True])
def test_gemm_variants(counts, K, N, dtype, wide):
    R = sum(counts)
    w = ref.experts(len(counts), N, K, R + N)
    x = torch.randn(R, K, generator=gen(R), device=DEV).to(dtype)
    out = check_gemm(x, by_counts(counts), w, out_dtype=F if wide else None)
    x[R // 2] = math.nan
    again = ffn.moe_gemm(x, by_counts(counts), w, out_dtype=F if wide else None)
    keep = torch.arange(R, device=DEV) != R // 2
    assert torch.isnan(again[R // 2]).all() and torch.equal(again[keep], out[keep])


@pytest.mark.parametrize("T,E,k,K,N", [(400, 4, 1, 96, 8192), (300, 4, 2, 160, 4128), (130, 3, 1, 288, 12000),
                                       (64, 64, 8, 96, 64), (600, 1, 1, 32, 64)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward_variants(T, E, k, K, N, dtype):
    ws = layer(E, K, N, T)
    x = torch.randn(T, K, generator=gen(T), device=DEV).to(dtype)
    ids = torch.randint(-1, E, (T, k), generator=gen(T + 1), device=DEV, dtype=torch.int32)
    p = torch.rand(T, k, generator=gen(T + 2), device=DEV)
    check_forward(x, ids, p, ws)
    ids[:] = E - 1  # one expert has all
    check_forward(x, ids, p, ws, ffn.ACT_GELU_TANH)


# Reductions past what a workgroup's registers hold, which go block by block: whole blocks, a last one of 64 columns
# and of others, several tiles of an expert, one weight row.
@pytest.mark.parametrize("K,N", [(5632, 96), (6080, 31), (6208, 33), (8192, 130), (10304, 1), (14336, 512), (14400, 95), (65536, 17)])
@pytest.mark.parametrize("counts", [[1], [0, 1, 16, 0, 3], [17, 0, 2, 33] + [0] * 4, [1] * 20 + [40]],
                         ids=lambda c: "_".join(map(str, c[:4])))
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gemm_reductions_in_blocks(counts, K, N, dtype):
    R = sum(counts)
    w = ref.experts(len(counts), N, K, R + N)
    x = torch.randn(R, K, generator=gen(R + K), device=DEV).to(dtype)
    out = check_gemm(x, by_counts(counts), w, out_dtype=F if N % 2 else None)
    x[R // 2, K - 1] = math.nan
    again = ffn.moe_gemm(x, by_counts(counts), w, out_dtype=F if N % 2 else None)
    keep = torch.arange(R, device=DEV) != R // 2
    assert torch.isnan(again[R // 2]).all() and torch.equal(again[keep], out[keep])


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (3, 3, 3), (40, 8, 2), (255, 40, 2), (300, 64, 3)])
@pytest.mark.parametrize("K,N", [(512, 14336), (5696, 6144), (8256, 160), (6208, 6272)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward_reductions_in_blocks(T, E, k, K, N, dtype):
    ws = layer(E, K, N, T)
    x = torch.randn(T, K, generator=gen(T), device=DEV).to(dtype)
    ids = torch.randint(-1, E, (T, k), generator=gen(T + 1), device=DEV, dtype=torch.int32)
    p = torch.rand(T, k, generator=gen(T + 2), device=DEV)
    check_forward(x, ids, p, ws)


def test_gemm_rows_outside_all_experts_are_left():
    w = ref.experts(3, 64, 128, 1)
    x = torch.randn(100, 128, generator=gen(2), device=DEV).to(BF)
    offsets = torch.tensor([10, 20, 20, 63], device=DEV, dtype=torch.int32)
    check_gemm(x, offsets, w)
    check_gemm(x, torch.zeros(4, device=DEV, dtype=torch.int32), w)


def test_gemm_offsets_and_rows_out_of_range_stay_inside():
    """Such values are a caller's mistake; nothing outside the buffers is read or written for them."""
    w = ref.experts(3, 64, 128, 1)
    x = torch.randn(50, 128, generator=gen(2), device=DEV).to(BF)
    room = torch.full((50 + 64, 64), -77.0, dtype=BF, device=DEV)
    for off in ([-5, 10, 2 ** 31 - 1, 7], [-(2 ** 31), 2 ** 31 - 1, 0, 50], [50, 40, 30, 20]):
        ffn.moe_gemm(x, torch.tensor(off, device=DEV, dtype=torch.int32), w, out=room[:50])
        assert (room[50:] == -77).all()
    many = ref.experts(1000, 64, 128, 1)  # every expert but the last claims all rows, or half of them do
    for off in ([0, 50] * 500 + [50], [0] * 500 + [50] * 501):
        ffn.moe_gemm(x, torch.tensor(off, device=DEV, dtype=torch.int32), many, out=room[:50])
        assert (room[50:] == -77).all()
    rows = torch.tensor([-1, 2 ** 31 - 1, 0, -(2 ** 31)] * 8, device=DEV, dtype=torch.int32)
    out = ffn.moe_gemm(x, torch.tensor([0, 10, 20, 32], device=DEV, dtype=torch.int32), w, rows=rows, top_k=3)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("m", [1, 20, 70, 200])
def test_gemm_special_values_stay_in_their_rows_and_channels(m):
    K, N = 288, 200
    w = ref.experts(2, N, K, 9)
    x = torch.randn(2 * m, K, generator=gen(m), device=DEV).to(BF)
    off = by_counts([m, m])
    clean = ffn.moe_gemm(x, off, w)
    bad = x.clone()
    bad[0, 5] = math.nan
    bad[m, 40] = math.inf
    out = ffn.moe_gemm(bad, off, w)
    assert torch.isnan(out[0]).all() and not torch.isfinite(out[m]).any()
    keep = [i for i in range(2 * m) if i not in (0, m)]
    assert torch.equal(out[keep], clean[keep])
    w.scales[1, 17, 3] = 0x7F  # a NaN scale
    out = ffn.moe_gemm(x, off, w)
    assert torch.isnan(out[m:, 17]).all()
    out[m:, 17] = clean[m:, 17]
    assert torch.equal(out, clean)


def test_gemm_every_code_and_scale():
    """All 256 bytes of codes against every finite E4M3 scale, one column at a time: exact products."""
    N = 254
    byte = torch.arange(256, device=DEV, dtype=torch.int32)
    scale = torch.cat([byte[:127], byte[128:255]]).to(torch.uint8)
    codes = byte.to(torch.uint8).repeat(N, 1).unsqueeze(0).contiguous()       # [1, 254, 512 / 2]
    scales = scale.view(N, 1).expand(N, 32).unsqueeze(0).contiguous()
    w = ffn.MoeDeviceWeight(codes, scales, torch.ones(1, device=DEV))
    for dtype in (BF, HF):
        x = torch.eye(512, device=DEV).to(dtype)
        out = ffn.moe_gemm(x, by_counts([512]), w, out_dtype=F)
        assert torch.equal(out.double(), ref.dense(w, 0).t())
        one = ffn.moe_gemm(x[7:8].contiguous(), by_counts([1]), w, out_dtype=F)
        assert torch.equal(one[0].double(), ref.dense(w, 0)[:, 7])


@pytest.mark.parametrize("m", [3, 50, 300])
def test_gemm_values_below_the_smallest_normal_one(m):
    """f16 rows of multiples of 2^-24 below 2^-14 keep their value, and so do such results: off by half a step of
    2^-24 beside the sum's own bound."""
    w = ref.experts(1, 96, 128, m)
    x = (torch.randint(-1000, 1001, (m, 128), generator=gen(m), device=DEV).double() * 2.0 ** -24).to(HF)
    y, b = ref.gemm(x, by_counts([m]), w)
    assert (y.abs() > 2.0 ** -20).any()
    out = ffn.moe_gemm(x, by_counts([m]), w, out_dtype=F)
    ref.within(out, y, b)
    out = ffn.moe_gemm(x, by_counts([m]), w)
    ref.within(out, y, b + (half(HF) * (y.abs() + b)).clamp_min(2.0 ** -25))


@pytest.mark.parametrize("T", [2, 300])
def test_forward_of_one_expert_that_all_tokens_name(T):
    """A router that has collapsed: many experts, all rows with a few of them."""
    ws = layer(96, 192, 128, T)
    x = torch.randn(T, 192, generator=gen(T), device=DEV).to(BF)
    ids = torch.tensor([[95, 3, 3]], device=DEV, dtype=torch.int32).repeat(T, 1)
    p = torch.rand(T, 3, generator=gen(T + 1), device=DEV)
    check_forward(x, ids, p, ws)


# ------------------------------------------------------------------- the layer


def layer(E, K, N, seed):
    return ref.experts(E, N, K, seed), ref.experts(E, N, K, seed + 1), ref.experts(E, K, N, seed + 2)


def check_forward(x, ids, p, ws, act=ffn.ACT_SILU):
    out = ffn.moe_forward(x, ids, p, *ws, act)
    ref.within(out, *ref.forward(x, ids, p, *ws, act))
    assert torch.equal(out, ffn.moe_forward(x, ids, p, *ws, act))
    return out


@pytest.mark.parametrize("T,E,k,K,N", [(1, 8, 2, 256, 512), (1, 1, 1, 32, 32), (2, 4, 4, 96, 160), (5, 64, 8, 352, 224),
                                       (17, 3, 2, 256, 128), (33, 128, 8, 512, 96), (64, 16, 4, 160, 288),
                                       (150, 2, 2, 288, 320), (300, 5, 3, 256, 256), (1, 8, 3, 5120, 2048),
                                       (9, 6, 2, 2048, 1024)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("act", [ffn.ACT_SILU, ffn.ACT_GELU_TANH])
def test_forward(T, E, k, K, N, dtype, act):
    g = gen(T + E)
    ws = layer(E, K, N, T)
    x = torch.randn(T, K, generator=g, device=DEV).to(dtype)
    p, ids = torch.softmax(torch.randn(T, E, generator=g, device=DEV), 1).topk(k, 1)
    ids = ids.int().contiguous()
    p = p.contiguous()
    check_forward(x, ids, p, ws, act)
    ids[torch.rand(T, k, generator=g, device=DEV) < 0.4] = -1
    check_forward(x, ids, p, ws, act)


def test_forward_without_experts_twice_the_same_and_out_of_range():
    ws = layer(4, 128, 96, 5)
    x = torch.randn(6, 128, generator=gen(5), device=DEV).to(BF)
    ids = torch.tensor([[-1, -1, -1], [2, 2, 2], [0, 4, 1], [-9, 3, 2 ** 30], [1, 0, 1], [3, 3, -1]], device=DEV, dtype=torch.int32)
    p = torch.rand(6, 3, generator=gen(6), device=DEV) - 0.3
    p[0] = math.nan  # (a slot without an expert adds nothing, whatever its weight)
    p[2, 1] = math.inf
    out = check_forward(x, ids, p, ws)
    assert (out[0] == 0).all()
    nobody = torch.full_like(ids, -1)
    assert (ffn.moe_forward(x, nobody, p, *ws) == 0).all()


@pytest.mark.parametrize("T", [1, 30, 200])
def test_forward_special_values_stay_in_their_token(T):
    ws = layer(5, 96, 128, 8)
    x = torch.randn(T, 96, generator=gen(8), device=DEV).to(BF)
    ids = torch.randint(0, 5, (T, 2), generator=gen(9), device=DEV, dtype=torch.int32)
    p = torch.rand(T, 2, generator=gen(9), device=DEV)
    clean = ffn.moe_forward(x, ids, p, *ws)
    x[T // 2, 3] = math.nan
    out = ffn.moe_forward(x, ids, p, *ws)
    assert torch.isnan(out[T // 2]).all()
    out[T // 2] = clean[T // 2]
    assert torch.equal(out, clean)
    w2 = ws[2].scale2.clone()
    ws[2].scale2[0] = math.nan  # an expert's own trouble
    x[T // 2, 3] = 0
    out = ffn.moe_forward(x, ids, p, *ws)
    with_it = (ids == 0).any(1)
    assert torch.isnan(out[with_it]).all() and torch.isfinite(out[~with_it]).all()
    ws[2].scale2.copy_(w2)


def test_forward_is_the_steps_it_is_made_of():
    """route, plan, product and the rest in a row give what the whole layer gives, within both sides' roundings."""
    T, E, k, K, N = 50, 12, 3, 256, 192
    ws = layer(E, K, N, 12)
    x = torch.randn(T, K, generator=gen(12), device=DEV).to(BF)
    ids, p = ffn.moe_route(torch.randn(T, E, generator=gen(13), device=DEV).to(BF), k)
    whole = check_forward(x, ids, p, ws)
    rows, offsets, places = ffn.moe_plan(ids, E)
    g = ffn.moe_gemm(x, offsets, ws[0], rows=rows, top_k=k, out_dtype=F)
    u = ffn.moe_gemm(x, offsets, ws[1], rows=rows, top_k=k, out_dtype=F)
    y = ffn.moe_gemm((torch.nn.functional.silu(g) * u).to(BF), offsets, ws[2])
    out = (y[places.long()].float() * p.unsqueeze(2)).sum(1)
    want, bound = ref.forward(x, ids, p, *ws, ffn.ACT_SILU)
    ref.within(out.to(BF), want, bound)
    ref.within(whole, want, bound)


# ------------------------------------------------- streams, graphs, buffers, sizes


def test_given_buffers_and_their_surroundings():
    """What is written is the outputs and no byte more."""
    T, E, k, K, N = 37, 6, 2, 160, 96
    ws = layer(E, K, N, 21)
    x = torch.randn(T, K, generator=gen(21), device=DEV).to(BF)
    ids, p = ffn.moe_route(torch.randn(T, E, generator=gen(22), device=DEV), k)
    need = ffn.moe_workspace_bytes(T, k, E, K, N)
    room = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    out = torch.full((T + 8, K), -77.0, dtype=BF, device=DEV)
    got = ffn.moe_forward(x, ids, p, *ws, out=out[4:4 + T], workspace=room[256:256 + need])
    assert torch.equal(got, ffn.moe_forward(x, ids, p, *ws))
    assert (out[:4] == -77).all() and (out[4 + T:] == -77).all()
    assert (room[:256] == 0x5A).all() and (room[256 + need:] == 0x5A).all()
    pad = torch.full((4 * 16384 + 64,), -5, dtype=torch.int32, device=DEV)
    ids = torch.randint(-1, E, (16384, 4), generator=gen(23), device=DEV, dtype=torch.int32)
    rows = pad[32:-32]
    ffn.moe_plan(ids, E, rows=rows)
    assert (pad[:32] == -5).all() and (pad[-32:] == -5).all()
    assert torch.equal(rows, ffn.moe_plan(ids, E)[0])


def test_another_stream():
    T, E, k, K, N = 64, 8, 2, 512, 256
    ws = layer(E, K, N, 31)
    x = torch.randn(T, K, generator=gen(31), device=DEV).to(BF)
    l = torch.randn(T, E, generator=gen(32), device=DEV)
    ids, p = ffn.moe_route(l, k)
    want = ffn.moe_forward(x, ids, p, *ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(5):
        outs = []
        for s in streams:
            i, q = ffn.moe_route(l, k, stream=s)
            outs.append(ffn.moe_forward(x, i, q, *ws, stream=s))
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, want)


@pytest.mark.parametrize("T", [1, 24, 300])
def test_graph_replays(T):
    """A recorded route + forward, replayed on new inputs with eager calls between the replays."""
    E, k, K, N = 8, 2, 256, 192
    ws = layer(E, K, N, 41)
    x = torch.randn(T, K, generator=gen(41), device=DEV).to(BF)
    l = torch.randn(T, E, generator=gen(42), device=DEV)

    def step():
        ids, p = ffn.moe_route(l, k)
        rows, offsets, _ = ffn.moe_plan(ids, E)
        return ffn.moe_forward(x, ids, p, *ws), ffn.moe_gemm(x, offsets, ws[0], rows=rows, top_k=k), offsets

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, y, offsets = step()
    for i in range(6):
        x.copy_(torch.randn(T, K, generator=gen(50 + i), device=DEV))
        l.copy_(torch.randn(T, E, generator=gen(60 + i), device=DEV))
        graph.replay()
        want, wy, _ = step()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert torch.equal(y[:int(offsets[-1])], wy[:int(offsets[-1])])


def test_two_graphs_share_a_workspace():
    T, E, k, K, N = 40, 8, 2, 256, 128
    ws = layer(E, K, N, 71)
    work = torch.empty(ffn.moe_workspace_bytes(T, k, E, K, N), dtype=torch.uint8, device=DEV)
    sets = []
    for i in range(2):
        x = torch.randn(T, K, generator=gen(72 + i), device=DEV).to(BF)
        ids, p = ffn.moe_route(torch.randn(T, E, generator=gen(74 + i), device=DEV), k)
        want = ffn.moe_forward(x, ids, p, *ws)
        out = torch.empty_like(want)
        ffn.moe_forward(x, ids, p, *ws, out=out, workspace=work)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ffn.moe_forward(x, ids, p, *ws, out=out, workspace=work)
        sets.append((graph, out, want, x, ids, p))
    for _ in range(4):
        for graph, out, *_ in sets:
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, out, want, *_ in sets:
            assert torch.equal(out, want)


def test_forward_captures_without_a_warm_call_of_its_shape():
    """The first call of a kernel sets it up; a later capture of another shape needs no call before it."""
    ws = layer(4, 128, 64, 81)
    x = torch.randn(3, 128, generator=gen(81), device=DEV).to(BF)
    ids = torch.tensor([[0, 1], [2, 3], [1, 1]], device=DEV, dtype=torch.int32)
    p = torch.rand(3, 2, generator=gen(82), device=DEV)
    want = ffn.moe_forward(x, ids, p, *ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ffn.moe_forward(x, ids, p, *ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.slow
def test_past_4_gib_of_weights_activations_and_outputs():
    # weights: the last expert's codes lie past 2^32 bytes
    E, N, K = 66, 4096, 32768
    codes = torch.randint(0, 256, (E, N, K // 2), device=DEV, dtype=torch.uint8, generator=gen(1))
    assert codes.numel() > 2 ** 32
    scales = torch.full((E, N, K // 16), 0x38, dtype=torch.uint8, device=DEV)
    w = ffn.MoeDeviceWeight(codes, scales, torch.full((E,), 2.0 ** -8, device=DEV))
    x = torch.randn(2, K, generator=gen(2), device=DEV).to(BF)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E] = 2
    check_gemm(x, off, w, out_dtype=F)
    del w, codes, scales
    # activations and outputs
    R = 70000
    w = ref.experts(2, 32, K, 3)
    x = torch.zeros(R, K, dtype=BF, device=DEV)
    assert x.numel() * 2 > 2 ** 32
    x[-130:] = torch.randn(130, K, generator=gen(4), device=DEV)
    out = ffn.moe_gemm(x, by_counts([R - 5, 5]), w, out_dtype=F)
    y, b = ref.gemm(x[-130:].contiguous(), by_counts([125, 5]), w)
    ref.within(out[-130:], y, b)
    assert (out[:-130] == 0).all()
    # tokens' rows read where they are, some of them past 2^32 bytes
    rows = torch.randint(3 * (R - 130), 3 * R, (200,), generator=gen(7), device=DEV, dtype=torch.int32)
    check_gemm(x, by_counts([150, 50]), w, rows=rows, top_k=3)
    check_gemm(x, by_counts([20, 3]), w, rows=rows[:23].contiguous(), top_k=3)
    del x, out
    N = 32768
    w = ref.experts(2, N, 32, 5)
    x = torch.randn(R, 32, generator=gen(6), device=DEV).to(BF)
    out = ffn.moe_gemm(x, by_counts([R - 5, 5]), w)
    assert out.numel() * 2 > 2 ** 32
    y, b = ref.gemm(x[-130:].contiguous(), by_counts([125, 5]), w)
    ref.within(out[-130:], y, b + half(BF) * (y.abs() + b))
    y, b = ref.gemm(x[:100].contiguous(), by_counts([100, 0]), w)
    ref.within(out[:100], y, b + half(BF) * (y.abs() + b))


@pytest.mark.parametrize("x_rows", [40000, 57000, 57400])
def test_tokens_rows_at_the_ends_of_32_bit_offsets(x_rows):
    # 2.6e9 bytes; a little under and over the 3.75e9 up to which rows are gathered with 32-bit offsets
    K = 32768
    w = ref.experts(2, 160, K, 3)
    x = torch.zeros(x_rows, K, dtype=HF, device=DEV)
    x[:30] = torch.randn(30, K, generator=gen(4), device=DEV)
    x[-30:] = torch.randn(30, K, generator=gen(5), device=DEV)
    rows = torch.randint(-60, 60, (200,), generator=gen(7), device=DEV, dtype=torch.int32)
    rows = torch.where(rows < 0, rows + 2 * x_rows, rows)
    check_gemm(x, by_counts([150, 50]), w, rows=rows, top_k=2)
    check_gemm(x, by_counts([20, 3]), w, rows=rows[:23].contiguous(), top_k=2)
