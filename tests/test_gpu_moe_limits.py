"""The sparse FFN's operators at the largest sizes that they take."""
import pytest
import torch

import moe_ref as ref
import w4a16_nvfp4_dense_amd as ffn
from moe_ref import DEV, gen

pytestmark = [pytest.mark.gpu, pytest.mark.slow]
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
T, E, k = 65536, 1024, 32


def choices(seed):
    ids = torch.randint(-20, E, (T, k), generator=gen(seed), device=DEV, dtype=torch.int32)
    return torch.where(ids < 0, -1, ids)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("with_bias", [False, True])
def test_choice(dtype, with_bias):
    logits = torch.randn(T, E, generator=gen(1), device=DEV).to(dtype)
    bias = torch.rand(E, generator=gen(2), device=DEV) if with_bias else None
    ids, w = ffn.moe_route(logits, k, ffn.SCORE_SIGMOID, bias=bias)
    score = 1 / (1 + torch.exp(-logits.double()))
    key = logits.double() if bias is None else score + bias.double()
    want = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids, want.int())
    s = score.gather(1, want)
    # in 32 bits: a score 5 U (exponential, sum, quotient), the sum of the chosen 6 more, their quotient and factor 3: 19 U
    assert ((w.double() - s / s.sum(1, keepdim=True)).abs() <= 20 * ref.U * w).all()


def test_order():
    ids = choices(3)
    rows, offsets, places = ffn.moe_plan(ids, E)
    flat = torch.where(ids < 0, E, ids).flatten()
    order = torch.sort(flat, stable=True).indices.int()
    real = int((flat < E).sum())
    assert torch.equal(rows[:real], order[:real]) and (rows[real:] == -1).all()
    assert torch.equal(offsets[1:], torch.bincount(flat, minlength=E + 1)[:E].cumsum(0).int()) and offsets[0] == 0
    want = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    want[order[:real].long()] = torch.arange(real, device=DEV, dtype=torch.int32)
    assert torch.equal(places.flatten(), want)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_layer(dtype):
    K, N = 64, 96
    ws = ref.experts(E, N, K, 4), ref.experts(E, N, K, 5), ref.experts(E, K, N, 6)
    x = torch.randn(T, K, generator=gen(7), device=DEV).to(dtype)
    ids, p = choices(8), torch.rand(T, k, generator=gen(9), device=DEV)
    out = ffn.moe_forward(x, ids, p, *ws)
    some = torch.cat([torch.arange(0, 70), torch.arange(T // 2, T // 2 + 70), torch.arange(T - 70, T)]).to(DEV)
    ref.within(out[some], *ref.forward(x[some], ids[some], p[some], *ws, ffn.ACT_SILU))


@pytest.mark.parametrize("counts", [[1, 0, 2], [40, 70]])
@pytest.mark.parametrize("out_dtype", [BF, F])
@pytest.mark.parametrize("N", [1 << 20, (1 << 20) - 1])
def test_channels(counts, out_dtype, N):
    w = ref.experts(len(counts), N, 32, 10)
    x = torch.randn(sum(counts), 32, generator=gen(11), device=DEV).to(BF)
    off = torch.tensor([0, *counts], device=DEV, dtype=torch.int32).cumsum(0).int()
    y, b = ref.gemm(x, off, w)
    if out_dtype == BF:
        b = b + ref.half(BF) * (y.abs() + b) + torch.finfo(BF).tiny
    ref.within(ffn.moe_gemm(x, off, w, out_dtype=out_dtype), y, b)


def test_rows_of_a_product():
    R = T * k
    w = ref.experts(E, 33, 32, 12)
    ids = choices(13)
    rows, off, _ = ffn.moe_plan(ids, E)
    x = torch.randn(T, 32, generator=gen(14), device=DEV).to(BF)
    out = torch.full((R, 33), -77.0, device=DEV)
    ffn.moe_gemm(x, off, w, rows=rows, top_k=k, out=out)
    y, b = ref.gemm(x, off, w, rows, k)
    real = int(off[E])
    ref.within(out[:real], y[:real], b[:real])
    assert (out[real:] == -77).all()


@pytest.mark.parametrize("K,N", [(65536, 32), (32, 65536), (65536, 4096)])
@pytest.mark.parametrize("rows", [1, 40])
def test_widths_of_a_layer(K, N, rows):
    ws = ref.experts(2, N, K, 15), ref.experts(2, N, K, 16), ref.experts(2, K, N, 17)
    x = torch.randn(rows, K, generator=gen(18), device=DEV).to(BF)
    ids = torch.randint(0, 2, (rows, 1), generator=gen(19), device=DEV, dtype=torch.int32)
    p = torch.rand(rows, 1, generator=gen(20), device=DEV)
    ref.within(ffn.moe_forward(x, ids, p, *ws), *ref.forward(x, ids, p, *ws, ffn.ACT_SILU))
