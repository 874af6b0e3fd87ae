"""Int8 products whose tiles are shared by several workgroups, where calls run beside each other and where a recorded
call is replayed again and again (needs an MI355X). The sums are exact, so everything is compared bit for bit."""
import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn
from test_gpu_int8 import _config, same_bits

pytestmark = pytest.mark.gpu

# tiles of every shape, shared ones among them: two parts of a tile, many parts, left-over tiles after whole rounds
SHAPES = [(1, 5120, 17408), (24, 4224, 1040), (64, 8192, 2048), (100, 5120, 5120), (300, 4112, 4096), (300, 2064, 17408),
          (2048, 528, 9232)]


def _needs_sharing(M, K, N):
    assert ffn.int8_gemm_workspace_bytes(M, K, N) > 0 or ffn.int8_gemm_workspace_bytes(M, N, K) > 0


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_many_streams_at_once(M, K, N):
    """Forwards and products on six streams, each with its own workspace: whichever launches hold which compute
    units, every tile is finished, with the same bits."""
    _needs_sharing(M, K, N)
    xq, xs, gate, up, down = _config(M, K, N, M + N)
    ref, prod = ffn.int8_forward(xq, xs, gate, up, down), ffn.int8_gemm(xq, xs, gate)
    streams = [torch.cuda.Stream() for _ in range(6)]
    ws = [torch.full((ffn.int8_workspace_bytes(M, K, N),), 0x5A, dtype=torch.uint8, device="cuda") for _ in streams]
    gws = [torch.full((max(16, ffn.int8_gemm_workspace_bytes(M, K, N)),), 0xA5, dtype=torch.uint8, device="cuda")
           for _ in streams]
    outs = [[(torch.empty_like(ref), torch.empty_like(prod)) for _ in range(4)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(4):
        for j, s in enumerate(streams):
            o, p = outs[j][i]
            ffn.int8_forward(xq, xs, gate, up, down, out=o, workspace=ws[j], stream=s)
            ffn.int8_gemm(xq, xs, gate, out=p, workspace=gws[j], stream=s)
    torch.cuda.synchronize()
    for o, p in (x for row in outs for x in row):
        assert same_bits(o, ref) and same_bits(p, prod)


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_replays_without_anything_between(M, K, N):
    """A recorded forward and product, replayed for one input after another with nothing but the replays writing the
    workspaces: what one replay leaves there must not pass for the next one's sums."""
    _needs_sharing(M, K, N)
    xq, xs, gate, up, down = _config(M, K, N, M + K)
    inputs = [(xq.roll(31 * i, 1).contiguous(), (xs * (1 + i)).contiguous()) for i in range(5)]
    refs = [(ffn.int8_forward(q, s, gate, up, down), ffn.int8_gemm(q, s, gate)) for q, s in inputs]
    q, s = inputs[0][0].clone(), inputs[0][1].clone()
    ws = torch.full((ffn.int8_workspace_bytes(M, K, N),), 0xFF, dtype=torch.uint8, device="cuda")
    gws = torch.full((max(16, ffn.int8_gemm_workspace_bytes(M, K, N)),), 0xFF, dtype=torch.uint8, device="cuda")
    out, prod = torch.empty_like(refs[0][0]), torch.empty_like(refs[0][1])

    def step():
        ffn.int8_forward(q, s, gate, up, down, out=out, workspace=ws)
        ffn.int8_gemm(q, s, gate, out=prod, workspace=gws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 1, 2, 3, 4, 1, 0, 3):
        q.copy_(inputs[i][0])
        s.copy_(inputs[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(out, refs[i][0]) and same_bits(prod, refs[i][1]), i
