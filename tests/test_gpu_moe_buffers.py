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


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_nothing_beside_the_buffers_is_written(T, E, k, K, N, dtype):
    """A workspace of just the bytes asked for, and an output, amid others' bytes; then one whose ids are all -1."""
    x, ids, p, ws = problem(T, E, k, K, N, 31, dtype)
    need = ffn.moe_workspace_bytes(T, k, E, K, N)
    room = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device=DEV)
    out = torch.full((T + 64, K), -77.0, dtype=dtype, device=DEV)
    for i in (ids, torch.full_like(ids, -1)):
        got = ffn.moe_forward(x, i, p, *ws, out=out[32:32 + T], workspace=room[4096:4096 + need])
        ref.within(got, *ref.forward(x, i, p, *ws, ffn.ACT_SILU))
        assert (out[:32] == -77).all() and (out[32 + T:] == -77).all()
        assert (room[:4096] == 0x5A).all() and (room[4096 + need:] == 0x5A).all()


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_plans_beside_others_bytes(T, E, k, K, N):
    _, ids, _, _ = problem(T, E, k, 32, 32, 41)
    ids[::3] = -1
    want = ffn.moe_plan(ids, E)
    need = ffn.moe_plan_workspace_bytes(T, k, E)
    room = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    outs = [torch.full((n + 128,), -5, dtype=torch.int32, device=DEV) for n in (T * k, E + 1, T * k)]
    rows, off, places = outs[0][64:-64], outs[1][64:-64], outs[2][64:-64].view(T, k)
    ffn.moe_plan(ids, E, rows=rows, offsets=off, places=places, workspace=room[256:256 + need] if need else None)
    for a, b in zip((rows, off, places), want):
        assert torch.equal(a, b)
    for o in outs:
        assert (o[:64] == -5).all() and (o[-64:] == -5).all()
    assert (room[:256] == 0x5A).all() and (room[256 + need:] == 0x5A).all()


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_several_streams_at_once(T, E, k, K, N):
    x, ids, p, ws = problem(T, E, k, K, N, 51)
    want = ffn.moe_forward(x, ids, p, *ws)
    plan = ffn.moe_plan(ids, E)
    ref.within(want, *ref.forward(x, ids, p, *ws, ffn.ACT_SILU))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(4):
        outs = [(ffn.moe_forward(x, ids, p, *ws, stream=s), ffn.moe_plan(ids, E, stream=s)) for s in streams]
        torch.cuda.synchronize()
        for o, pl in outs:
            assert torch.equal(o, want)
            assert all(torch.equal(a, b) for a, b in zip(pl, plan))


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_graphs_that_share_a_workspace(T, E, k, K, N):
    """Two recorded calls of different shapes on one workspace, replayed in turn on changing inputs, with eager calls on
    the same workspace between them."""
    work = torch.empty(ffn.moe_workspace_bytes(T, k, E, K, N), dtype=torch.uint8, device=DEV)
    sets = []
    for i, t in enumerate((T, T - T // 5)):
        x, ids, p, ws = problem(t, E, k, K, N, 61 + 7 * i)
        out = torch.empty_like(x)
        ffn.moe_forward(x, ids, p, *ws, out=out, workspace=work)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ffn.moe_forward(x, ids, p, *ws, out=out, workspace=work)
        sets.append((graph, out, x, ids, p, ws))
    for i in range(4):
        for j, (_, out, x, ids, p, _) in enumerate(sets):
            x.copy_(torch.randn(x.shape, generator=gen(80 + i), device=DEV))
            fresh, q = ffn.moe_route(torch.randn(x.shape[0], E, generator=gen(90 + 2 * i + j), device=DEV), k)
            ids.copy_(fresh)
            p.copy_(q)
            out.zero_()
        for graph, *_ in sets:
            graph.replay()
        if i % 2:
            graph.replay()
        torch.cuda.synchronize()
        for _, out, x, ids, p, ws in sets:
            assert torch.equal(out, ffn.moe_forward(x, ids, p, *ws, workspace=work))


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_the_whole_step_recorded(T, E, k, K, N):
    """Choice, order, product and layer in one graph, replayed on new logits and inputs."""
    x, _, _, ws = problem(T, E, k, K, N, 101)
    logits = torch.randn(T, E, generator=gen(102), device=DEV)

    def step():
        ids, p = ffn.moe_route(logits, k)
        rows, off, places = ffn.moe_plan(ids, E)
        return ids, p, rows, off, places, ffn.moe_gemm(x, off, ws[0], rows=rows, top_k=k), ffn.moe_forward(x, ids, p, *ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        recorded = step()
    for i in range(5):
        x.copy_(torch.randn(T, K, generator=gen(110 + i), device=DEV))
        logits.copy_(torch.randn(T, E, generator=gen(120 + i), device=DEV))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for a, b in zip(recorded, eager):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,E,k,K,N", SIZES)
def test_a_shape_first_seen_by_a_capture(T, E, k, K, N):
    """The kernels have run before, on another number of tokens; this one runs for the first time in a replay."""
    x, ids, p, ws = problem(T, E, k, K, N, 131)
    ffn.moe_forward(x, ids, p, *ws)
    t = T - 3
    y, i, q = x[3:].clone(), ids[3:].flip(0).contiguous(), p[3:].contiguous()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ffn.moe_forward(y, i, q, *ws)
    assert out.shape == (t, K)
    for n in range(3):
        y.copy_(torch.randn(t, K, generator=gen(140 + n), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        ref.within(out, *ref.forward(y, i, q, *ws, ffn.ACT_SILU))
