"""Buffers, streams and graphs of the sparse FFN, at sizes that take each of its ways: without a plan (up to 512 slots),
with one launch of it, and with two (more than 8192 slots)."""
import pytest
import torch

import moe_ref as ref
import w4a16_nvfp4_dense_amd as ffn
from moe_ref import DEV, gen

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32

# tokens, experts, top_k, K, N: 74 slots; 800 and 2100, tiles of 32 and 64 rows; 12000, of 128, and plans of two launches
SIZES = [(37, 6, 2, 160, 96), (400, 40, 2, 160, 96), (700, 30, 3, 288, 160), (3000, 24, 4, 160, 352)]


def problem(T, E, k, K, N, seed, dtype=BF):
    ws = ref.experts(E, N, K, seed), ref.experts(E, N, K, seed + 1), ref.experts(E, K, N, seed + 2)
    x = torch.randn(T, K, generator=gen(seed), device=DEV).to(dtype)
    ids, p = ffn.moe_route(torch.randn(T, E, generator=gen(seed + 1), device=DEV), k)
    return x, ids, p, ws


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_in_place(T, E, k, K, N):
    x, ids, p, ws = problem(T, E, k, K, N, 11)
    want = ffn.moe_forward(x, ids, p, *ws)
    ref.within(want, *ref.forward(x, ids, p, *ws, ffn.ACT_SILU))
    assert ffn.moe_forward(x, ids, p, *ws, out=x) is x
    assert torch.equal(x, want)


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_buffers_that_touch(T, E, k, K, N):
    """Inputs and outputs end to end in one piece of memory do not overlap, and one weight may be gate and up."""
    x, ids, p, ws = problem(T, E, k, K, N, 21)
    one = ws[0], ws[0], ws[2]
    need = ffn.moe_workspace_bytes(T, k, E, K, N)
    want = ffn.moe_forward(x, ids, p, *one)
    size = T * K * 2
    room = torch.zeros(3 * size + need, dtype=torch.uint8, device=DEV)
    at = [0, size, size + need, 2 * size + need]
    first, work, out = room[:size].view(BF).view(T, K), room[at[1]:at[2]], room[at[2]:at[3]].view(BF).view(T, K)
    first.copy_(x)
    ffn.moe_forward(first, ids, p, *one, out=out, workspace=work)
    assert torch.equal(out, want) and torch.equal(first, x)
    with pytest.raises(ffn.FfnError, match="overlap"):
        ffn.moe_forward(first, ids, p, *one, out=room[16:16 + size].view(BF).view(T, K), workspace=work)
