"""Products grouped by expert whose sums are exact in fp32, in whatever order they are added: every one of the kernels'
ways (chunks of a wave, groups of waves, blocks, tiles, 64-bit addresses) has to give the very number. A column left out,
taken twice or multiplied with another's scale shows, however long the reduction is."""
import pytest
import torch

import moe_ref as ref
import w4a16_nvfp4_dense_amd as ffn
from moe_ref import DEV, gen

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def whole(E, rows, cols, seed):
    """Experts of random codes, block scales of 0.5, 1 and 2 and of both signs, and scale2 of powers of two: products
    with -1, 0 and 1 are multiples of a quarter up to 12, so sums of 65536 are below 2^22 of them, exact."""
    g = gen(seed)
    codes = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device=DEV, dtype=torch.uint8)
    kinds = torch.tensor([0x30, 0x38, 0x40, 0xB0, 0xB8, 0xC0], device=DEV, dtype=torch.uint8)
    scales = kinds[torch.randint(0, 6, (E, rows, cols // 16), generator=g, device=DEV)]
    scale2 = 2.0 ** torch.randint(-9, 3, (E,), generator=g, device=DEV).float()
    return ffn.MoeDeviceWeight(codes, scales, scale2)


def signs(rows, cols, seed, dtype):
    return torch.randint(-1, 2, (rows, cols), generator=gen(seed), device=DEV).to(dtype)


def offsets(counts):
    return torch.tensor([0, *counts], device=DEV, dtype=torch.int32).cumsum(0).int()


def check(counts, K, N, dtype, top_k=0):
    E, R = len(counts), sum(counts)
    w, off = whole(E, N, K, R + K + N), offsets(counts)
    rows = None
    if top_k:
        T = (R + top_k - 1) // top_k
        rows = torch.randperm(T * top_k, generator=gen(R), device=DEV)[:R].int()
        x = signs(T, K, K, dtype)
    else:
        x = signs(R, K, K, dtype)
    want, _ = ref.gemm(x, off, w, rows, top_k or 1)
    wide = ffn.moe_gemm(x, off, w, rows=rows, top_k=top_k or 1, out_dtype=F)
    assert torch.equal(wide.double(), want)
    # (one rounding, to the nearest; f16 ends at 65504, which 12 * 65536 * 4 may pass and its rounding makes infinite)
    assert torch.equal(ffn.moe_gemm(x, off, w, rows=rows, top_k=top_k or 1), want.float().to(dtype))


FEW = [1, 0, 3, 2, 17, 1, 5, 0]                        # tiles of 16 rows: one of a row, none, a second of one row
MANY = (FEW + [1] * 8) * 4                             # 64 experts, 148 rows: passes for every compute unit


# Reductions of one to six chunks of a wave, at their ends and not of whole chunks; up to 1024 columns with enough passes
# two groups of four waves instead (MANY), with a last group of no channels, of one, and full; past 6144 blocks.
@pytest.mark.parametrize("K", [32, 480, 512, 544, 800, 992, 1024, 1056, 2048, 2080, 2560, 3040, 3104, 4096, 4128, 5120, 5152,
                               6080, 6144, 6208, 8192, 10304, 65536])
@pytest.mark.parametrize("N", [1, 31, 97])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_few_rows(K, N, dtype):
    check(FEW, K, N, dtype)
    check(FEW, K, N, dtype, top_k=3)
    check([16] * 4, K, N, dtype)


@pytest.mark.parametrize("K", [288, 512, 544, 736, 800, 992, 1024])
@pytest.mark.parametrize("N", [897, 928, 960, 993, 1024])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_two_groups_of_waves(K, N, dtype):
    check(MANY, K, N, dtype)
    check(MANY, K, N, dtype, top_k=2)


# Tiles of 32, 64 and 128 rows, of 128 and 256 channels: whole and part stages of the reduction, tails of rows and channels.
@pytest.mark.parametrize("counts,N", [([20, 31, 1, 17, 18], 513), ([40, 64, 31, 50], 300), ([40, 64, 31, 50], 16501),
                                      ([70, 128, 1, 97], 130), ([200, 129, 33, 300], 8193), ([64, 65, 129, 257], 9000)])
@pytest.mark.parametrize("K", [32, 96, 160, 512, 672, 4128])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_tiles(counts, K, N, dtype):
    check(counts, K, N, dtype)
    check(counts, K, N, dtype, top_k=4)


@pytest.mark.parametrize("counts", [[1], [130], [33, 0, 70]])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_tiles_of_the_longest_reductions(counts, dtype):
    check(counts + [200], 65536, 33, dtype)


@pytest.mark.slow
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("K", [32768, 32800, 32864])
def test_rows_past_32_bit_offsets(K, dtype):
    """Tokens' rows gathered through 64-bit addresses; a last stage of 32 and of 96 columns."""
    T = 57400
    assert T * K * 2 >= 0xE0000000
    x = torch.zeros(T, K, dtype=dtype, device=DEV)
    x[:40], x[-40:] = signs(40, K, 1, dtype), signs(40, K, 2, dtype)
    w = whole(3, 161, K, 3)
    slot = torch.randint(-120, 120, (230,), generator=gen(4), device=DEV)
    rows = torch.where(slot < 0, slot + 3 * T, slot).int()
    for counts in ([150, 17, 63], [70, 1, 90]):
        off, n = offsets(counts), sum(counts)
        want, _ = ref.gemm(x, off, w, rows[:n], 3)
        out = ffn.moe_gemm(x, off, w, rows=rows[:n].contiguous(), top_k=3, out_dtype=F)
        assert torch.equal(out.double(), want)


# ------------------------------------------------------------------- the layer


def layer(E, K, N, seed):
    return ref.experts(E, N, K, seed), ref.experts(E, N, K, seed + 1), ref.experts(E, K, N, seed + 2)


def check_forward(T, E, k, K, N, dtype):
    ws = layer(E, K, N, T)
    x = torch.randn(T, K, generator=gen(T), device=DEV).to(dtype)
    ids = torch.randint(-1, E, (T, k), generator=gen(T + 1), device=DEV, dtype=torch.int32)
    p = torch.rand(T, k, generator=gen(T + 2), device=DEV)
    for act in (ffn.ACT_SILU, ffn.ACT_GELU_TANH):
        out = ffn.moe_forward(x, ids, p, *ws, act)
        ref.within(out, *ref.forward(x, ids, p, *ws, act))


# gate and up, down, or both in two groups of waves; without a plan (up to 512 slots) and with one
@pytest.mark.parametrize("T,E,k", [(70, 96, 2), (300, 96, 2), (500, 64, 2)])
@pytest.mark.parametrize("K,N", [(800, 512), (544, 544), (1024, 992), (992, 1024)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward_in_two_groups_of_waves(T, E, k, K, N, dtype):
    check_forward(T, E, k, K, N, dtype)


@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (40, 8, 2), (300, 40, 2)])
@pytest.mark.parametrize("K,N", [(2080, 3104), (2560, 4096), (4096, 2560), (1056, 2080), (5120, 5152)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward_of_three_to_six_chunks(T, E, k, K, N, dtype):
    check_forward(T, E, k, K, N, dtype)


@pytest.mark.slow
@pytest.mark.parametrize("dtype", [BF, HF])
def test_forward_of_tokens_past_32_bit_offsets(dtype):
    """All but the first and the last tokens without an expert, as padding is."""
    T, E, k, K, N = 65536, 3, 1, 28704, 96
    assert T * K * 2 >= 0xE0000000
    ws = layer(E, K, N, 5)
    some = torch.cat([torch.arange(0, 90), torch.arange(T - 130, T)]).to(DEV)
    x = torch.zeros(T, K, dtype=dtype, device=DEV)
    x[some] = torch.randn(len(some), K, generator=gen(6), device=DEV).to(dtype)
    ids = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    ids[some] = torch.randint(0, E, (len(some), k), generator=gen(7), device=DEV, dtype=torch.int32)
    p = torch.rand(T, k, generator=gen(8), device=DEV)
    out = ffn.moe_forward(x, ids, p, *ws)
    ref.within(out[some], *ref.forward(x[some], ids[some], p[some], *ws, ffn.ACT_SILU))
    out[some] = 0
    assert not out.any()


@pytest.mark.parametrize("T", [1, 30, 200])
def test_h_past_the_range_of_f16(T):
    """|h| above 65504 is infinite in f16 and its token's outputs with it, no other's; in bf16 it is in range."""
    E, K, N = 3, 96, 128
    ws = layer(E, K, N, 9)
    x = torch.randn(T, K, generator=gen(10), device=DEV)
    ids = torch.randint(0, E, (T, 2), generator=gen(11), device=DEV, dtype=torch.int32)
    p = torch.rand(T, 2, generator=gen(12), device=DEV)
    loud = T // 2
    clean = ffn.moe_forward(x.to(HF), ids, p, *ws)
    x[loud] *= 4000
    out = ffn.moe_forward(x.to(HF), ids, p, *ws)
    assert not torch.isfinite(out[loud]).any()
    out[loud] = clean[loud]
    assert torch.equal(out, clean)
    x = x.to(BF)
    ref.within(ffn.moe_forward(x, ids, p, *ws), *ref.forward(x, ids, p, *ws, ffn.ACT_SILU))
