"""The FFN half of a stack of decoder layers on the int8 operators.

    python examples/int8_block.py [--layers L] [--hidden K] [--inter N] [--tokens M] [--steps S]

Each layer is norm -> gated FFN, added to the residual stream:

    t = t + delta;  delta = W_d q(act(W_g n) * (W_u n)),  n = q(norm(t))

NVFP4 weights become int8 rows once (``int8_prepare_weight``). A step is then two calls a layer:
``int8_rmsnorm`` adds the layer before's output to the residual stream, norms it and quantises it in one pass,
and ``int8_forward`` runs the FFN on the codes. The buffers are allocated once, and a step is recorded as a HIP
graph, as a decoding loop would do. The result is compared with the same layers on the W4A16 path."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_nvfp4_dense_amd as ffn  # noqa: E402

EPS = 1e-6


def make_layers(layers, K, N, seed=0, device="cuda"):
    """Random layers of a trained model's scale: (norm weight, NVFP4 gate, up, down)."""
    g = torch.Generator(device=device).manual_seed(seed)

    def weight(rows, cols):
        w = torch.randn(rows, cols, generator=g, device=device) / cols ** 0.5
        return ffn.quantize_weight(w.to(torch.bfloat16))

    return [(1.0 + 0.1 * torch.randn(K, generator=g, device=device), weight(N, K), weight(N, K), weight(K, N))
            for _ in range(layers)]


class Int8Stack:
    """The layers on int8 weights, with every buffer that a step of M tokens needs."""

    def __init__(self, layers, M, act=ffn.ACT_SILU):
        self.layers = [(norm, *(ffn.int8_prepare_weight(w) for w in weights)) for norm, *weights in layers]
        N, K = self.layers[0][1].rows, self.layers[0][1].cols
        dev = self.layers[0][0].device
        self.act = act
        self.codes = torch.empty(M, K, dtype=torch.int8, device=dev)
        self.scales = torch.empty(M, dtype=torch.float32, device=dev)
        self.delta = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        self.stream = torch.empty(M, K, dtype=torch.bfloat16, device=dev)  # the residual stream
        self.workspace = torch.empty(ffn.int8_workspace_bytes(M, K, N), dtype=torch.uint8, device=dev)

    def step(self, x):
        """The residual stream after all layers, for the hidden states x (bf16 [M, K])."""
        for i, (norm, gate, up, down) in enumerate(self.layers):
            ffn.int8_rmsnorm(x if i == 0 else self.delta, norm, EPS, residual=None if i == 0 else self.stream,
                             codes=self.codes, scales=self.scales, sum_out=self.stream)
            ffn.int8_forward(self.codes, self.scales, gate, up, down, self.act, out=self.delta,
                             workspace=self.workspace)
        return self.stream + self.delta


def w4a16_step(layers, x, act=ffn.ACT_SILU):
    """The same layers on the W4A16 path, the norm in torch."""
    t = x
    for norm, gate, up, down in layers:
        f = t.float()
        n = (f * torch.rsqrt(f.pow(2).mean(1, keepdim=True) + EPS) * norm).to(torch.bfloat16)
        t = t + ffn.forward(n, gate, up, down, act)
    return t


def capture(stack, x):
    """(graph, output): a replay of the graph runs a step on what x holds then."""
    stack.step(x)  # first use sets up the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stack.step(x)
    return graph, out


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--hidden", type=int, default=5120)
    p.add_argument("--inter", type=int, default=17408)
    p.add_argument("--tokens", type=int, default=1)
    p.add_argument("--steps", type=int, default=50)
    o = p.parse_args()
    layers = make_layers(o.layers, o.hidden, o.inter)
    x = torch.randn(o.tokens, o.hidden, device="cuda").to(torch.bfloat16)
    stack = Int8Stack(layers, o.tokens)
    graph, out = capture(stack, x)
    graph.replay()
    ref = w4a16_step(layers, x).double() - x.double()
    got = out.double() - x.double()
    error = float((got - ref).norm() / ref.norm())
    print(f"{o.layers} layers, {o.hidden}/{o.inter}, {o.tokens} tokens: what the layers add differs from the W4A16 "
          f"path by {100 * error:.2f}%", flush=True)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(o.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{1000 * begin.elapsed_time(end) / o.steps / o.layers:.1f} us a layer", flush=True)


if __name__ == "__main__":
    main()
