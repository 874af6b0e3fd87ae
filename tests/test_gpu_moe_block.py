"""The example that runs the sparse FFN's operators together: its step against the dense FFN, expert by expert, and its
graph against its eager step."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("moe_block", _PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("M", [1, 6, 70])
def test_block(block, M):
    """One layer, so that both sides choose the same experts. A rounding to bf16 is off by at most 2^-8 of the value:
    the residual sums' on either side come to 2 * 2^-8 of the stream, the deltas' to 2 * 2^-8 of them, the dense
    FFN's own outputs' to 2^-8 of sum_j p_j |y_j|, and sums of another order move some h by a step, 2^-7 of it,
    which its product with W_d carries as such. For top_k = 3 independent outputs sum_j p_j |y_j| is about sqrt(3)
    times their sum, under 2 sqrt(3)."""
    layers = block.make_layers(1, 8, 512, 256, seed=M)
    g = torch.Generator(device="cuda").manual_seed(100 + M)
    t = torch.randn(M, 512, generator=g, device="cuda").to(torch.bfloat16)
    stack = block.SparseStack(layers, M, 3)
    got = stack.step(t).double()
    ref = block.dense_step(layers, t, 3).double()
    moved = (ref - t.double()).norm()
    assert (got - ref).norm() < 2 ** -7 * ref.norm() + (2 ** -7 + (2 ** -8 + 2 ** -7) * 2 * 3 ** 0.5) * moved


@pytest.mark.parametrize("M", [1, 6, 70])
def test_graph(block, M):
    layers = block.make_layers(2, 8, 256, 320, seed=M)
    g = torch.Generator(device="cuda").manual_seed(200 + M)
    t = torch.randn(M, 256, generator=g, device="cuda").to(torch.bfloat16)
    stack = block.SparseStack(layers, M, 2)
    graph, out = block.capture(stack, t)
    for i in range(4):
        fresh = torch.randn(M, 256, generator=g, device="cuda").to(torch.bfloat16)
        eager = stack.step(fresh).clone()
        t.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
