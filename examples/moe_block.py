"""The FFN half of a stack of sparse (mixture of experts) decoder layers.

    python examples/moe_block.py [--layers L] [--hidden K] [--inter N] [--experts E] [--top-k k] [--tokens M] [--steps S]

Each layer is norm -> router -> sparse FFN, added to the residual stream:

    t = t + delta;  delta = sum_j p_j W_d,e (act(W_g,e n) * (W_u,e n)),  n = norm(t),  (e, p) = route(W_r n)

``moe_route`` chooses each token's experts and ``moe_forward`` runs them over their NVFP4 weights. The buffers are
allocated once, and a step is recorded as a HIP graph, as a decoding loop would do; the tokens' experts differ from
replay to replay. The result is compared with the same experts run one after another through the dense FFN."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_nvfp4_dense_amd as ffn  # noqa: E402

EPS = 1e-6


def make_layers(layers, experts, K, N, seed=0, device="cuda"):
    """Random layers of a trained model's scale: (norm weight, router weight, NVFP4 gate, up, down of each expert)."""
    g = torch.Generator(device=device).manual_seed(seed)

    def weights(rows, cols):
        return [ffn.quantize_weight((torch.randn(rows, cols, generator=g, device=device) / cols ** 0.5).to(torch.bfloat16))
                for _ in range(experts)]

    return [(1.0 + 0.1 * torch.randn(K, generator=g, device=device),
             (torch.randn(experts, K, generator=g, device=device) / K ** 0.5).to(torch.bfloat16),
             weights(N, K), weights(N, K), weights(K, N)) for _ in range(layers)]


def norm(t, weight):
    f = t.float()
    return (f * torch.rsqrt(f.pow(2).mean(1, keepdim=True) + EPS) * weight).to(torch.bfloat16)


class SparseStack:
    """The layers on stacked experts, with every buffer that a step of M tokens needs."""

    def __init__(self, layers, M, top_k, act=ffn.ACT_SILU):
        self.layers = [(n, r, *(ffn.MoeDeviceWeight.stack(w) for w in weights)) for n, r, *weights in layers]
        gate = self.layers[0][2]
        E, N, K = gate.experts, gate.rows, gate.cols
        dev = gate.codes.device
        self.act, self.top_k = act, top_k
        self.ids = torch.empty(M, top_k, dtype=torch.int32, device=dev)
        self.weights = torch.empty(M, top_k, dtype=torch.float32, device=dev)
        self.delta = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        self.workspace = torch.empty(ffn.moe_workspace_bytes(M, top_k, E, K, N), dtype=torch.uint8, device=dev)

    def step(self, t):
        """The residual stream after all layers, for t (bf16 [M, K])."""
        for weight, router, gate, up, down in self.layers:
            n = norm(t, weight)
            ffn.moe_route(n @ router.t(), self.top_k, ids=self.ids, weights=self.weights)
            ffn.moe_forward(n, self.ids, self.weights, gate, up, down, self.act, out=self.delta,
                            workspace=self.workspace)
            t = t + self.delta
        return t


def dense_step(layers, t, top_k, act=ffn.ACT_SILU):
    """The same layers, each expert's tokens through the dense FFN."""
    for weight, router, gate, up, down in layers:
        n = norm(t, weight)
        ids, p = ffn.moe_route(n @ router.t(), top_k)
        delta = torch.zeros(t.shape, device=t.device)
        for e in range(len(gate)):
            token, j = torch.nonzero(ids == e, as_tuple=True)
            if token.numel():
                y = ffn.forward(n[token].contiguous(), gate[e], up[e], down[e], act)
                delta[token] += y.float() * p[token, j].unsqueeze(1)
        t = t + delta.to(torch.bfloat16)
    return t


def capture(stack, t):
    """(graph, output): a replay of the graph runs a step on what t holds then."""
    stack.step(t)  # first use sets up the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stack.step(t)
    return graph, out


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--inter", type=int, default=1024)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--top-k", type=int, default=4)
    p.add_argument("--tokens", type=int, default=4)
    p.add_argument("--steps", type=int, default=50)
    o = p.parse_args()
    layers = make_layers(o.layers, o.experts, o.hidden, o.inter)
    t = torch.randn(o.tokens, o.hidden, device="cuda").to(torch.bfloat16)
    stack = SparseStack(layers, o.tokens, o.top_k)
    graph, out = capture(stack, t)
    graph.replay()
    ref = dense_step(layers, t, o.top_k).double() - t.double()
    got = out.double() - t.double()
    error = float((got - ref).norm() / ref.norm())
    print(f"{o.layers} layers, {o.hidden}/{o.inter}, {o.experts} experts, {o.top_k} of them for each of {o.tokens} "
          f"tokens: what the layers add differs from the dense FFN's by {100 * error:.2f}%", flush=True)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(o.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{1000 * begin.elapsed_time(end) / o.steps / o.layers:.1f} us a layer", flush=True)


if __name__ == "__main__":
    main()
