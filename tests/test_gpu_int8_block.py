"""The example that runs the int8 operators together: its step against the W4A16 path and its graph against
its eager step."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "int8_block.py")


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("int8_block", _PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("M", [1, 5, 48])
def test_block(block, M):
    """Rounding to 127 steps of a row's largest value leaves an error of s / sqrt(12) on each value. For about
    normal rows of up to 1024 values the largest is under 4.5 standard deviations, so 4.5 / 127 / sqrt(12) = 1.0%
    for a normed row or a weight; h, a product of two normals with a gate, has a largest value under 15 of its
    standard deviations: 3.4%. Relative errors of the operands of one product add in squares: gate and up sqrt(2) *
    1.0% each, carried through the gate's product by a factor under 2 in all, then 3.4% and 1.0%: under 5% a layer;
    of two layers, the second's input differs by less than the first's share: under 10% in all."""
    layers = block.make_layers(2, 512, 1024, seed=M)
    g = torch.Generator(device="cuda").manual_seed(100 + M)
    x = torch.randn(M, 512, generator=g, device="cuda").to(torch.bfloat16)
    stack = block.Int8Stack(layers, M)
    got = stack.step(x)
    ref = block.w4a16_step(layers, x)
    moved = ref.double() - x.double()
    assert float((got.double() - ref.double()).norm() / moved.norm()) < 0.10

    graph, out = block.capture(stack, x)
    for i in range(3):
        fresh = torch.randn(M, 512, generator=g, device="cuda").to(torch.bfloat16)
        eager = stack.step(fresh).clone()
        x.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
