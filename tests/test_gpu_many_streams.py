"""Forwards whose reductions are split over workgroups, beside each other on many streams and replayed with nothing
in between (needs an MI355X): whichever launches hold which compute units, and whatever one call leaves in a
workspace, every result has the bits of a call on its own."""
import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn

pytestmark = pytest.mark.gpu

ARMS = {}


def arm(name, M, K, N):
    """A forward of M tokens by its name: (workspace bytes, call(x, weights, out, workspace, stream))."""
    def add(f):
        ARMS[name] = (M, K, N, f)
        return f
    return add


def _w4a16(M, K, N):
    return ffn.workspace_bytes(M, K, N), lambda w: w, ffn.forward


arm("small_m16", 16, 5120, 17408)(_w4a16)       # small-batch arm, down product in 4 parts
arm("small_m17", 17, 5120, 17408)(_w4a16)       # both products in parts
arm("small_m40", 40, 5120, 17408)(_w4a16)       # three and six parts
arm("small_m33_short", 33, 5376, 2048)(_w4a16)


arm("prefill_m64", 64, 5120, 17408)(_w4a16)     # 128-row arm: the dual product finishes its split tiles in the launch
arm("prefill_m128", 128, 5120, 17408)(_w4a16)
arm("prefill_m41_short", 41, 2048, 1088)(_w4a16)   # many pieces of a tile
arm("prefill_m200", 200, 1024, 8256)(_w4a16)    # two blocks on the same words


def _fp4(M, K, N):
    """All three projections on 4 bits: the down product's reduction is split in parts."""
    return (ffn.w4a4_fp4_workspace_bytes(M, K, N), lambda w: [ffn.w4a4_prepare_weight(v) for v in w],
            ffn.w4a4_forward_fp4)


arm("fp4_m128", 128, 5120, 17408)(_fp4)
arm("fp4_m40_eight_parts", 40, 1024, 4096)(_fp4)
arm("fp4_m200", 200, 2048, 4096)(_fp4)  # two launches on the same words


@pytest.fixture(scope="module", params=list(ARMS))
def case(request):
    M, K, N, make = ARMS[request.param]
    need, prepare, call = make(M, K, N)
    g = torch.Generator(device="cuda").manual_seed(M + K)

    def weight(r, c):
        return ffn.quantize_weight((torch.randn(r, c, generator=g, device="cuda") / c ** 0.5).to(torch.bfloat16))

    weights = prepare((weight(N, K), weight(N, K), weight(K, N)))
    xs = [torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]
    refs = [call(x, *weights) for x in xs]
    torch.cuda.synchronize()
    return need, weights, call, xs, refs


def test_many_streams_at_once(case):
    need, weights, call, xs, refs = case
    streams = [torch.cuda.Stream() for _ in range(6)]
    spaces = [torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [[torch.empty_like(r) for r in refs] for _ in streams]
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        for s, ws, out in zip(streams, spaces, outs):
            call(x, *weights, out=out[i], workspace=ws, stream=s)
    torch.cuda.synchronize()
    for out in outs:
        for o, r in zip(out, refs):
            assert torch.equal(o.view(torch.int16), r.view(torch.int16))


def test_replays_without_anything_between(case):
    need, weights, call, xs, refs = case
    x, out = xs[0].clone(), torch.empty_like(refs[0])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    call(x, *weights, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, *weights, out=out, workspace=ws)
    for i in (0, 1, 2, 3, 1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), refs[i].view(torch.int16)), i
