"""Tensors that a binding makes for a call on a stream other than the current one come from that stream's memory, and
are marked as used on the current one. (From the current stream's pool they could be memory that kernels enqueued
there before still read: the call's stream does not wait for those.) The first part runs on the CPU, with stand-ins
for tensors and streams and calls of no tokens, which launch nothing; the second needs an MI355X."""
import contextlib

import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn
from test_binding_host import Fake

K, N = 256, 512
BF, F, I8, U8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8


class At(Fake):
    """A stand-in with an address, which an empty call never touches."""

    made = None

    def data_ptr(self):
        return 0x7F0000000000

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    def record_stream(self, s):
        self.recorded.append(s)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def nv(r, c):
    return ffn.DeviceWeight(At((r, c // 2)), At((r, c // 16)), 1.0)


def f8(r, c):
    return ffn.Fp8DeviceWeight(At((r, c)), At(((r + 127) // 128, (c + 127) // 128), F))


def mx(r, c):
    return ffn.MxDeviceWeight(At((r, c // 2)), At((r, c // 32)), 1.0)


def i8(r, c):
    return ffn.Int8DeviceWeight(At((r, c), I8), At((r,), F))


x, xq, xs = At((0, K), BF), At((0, K), I8), At((0,), F)
ga, ua = At((0, N), F), At((0, N), F)
CALLS = {
    "forward": (2, lambda s: ffn.forward(x, nv(N, K), nv(N, K), nv(K, N), stream=s)),
    "dual_gemv": (2, lambda s: ffn.dual_gemv(x, nv(N, K), nv(N, K), stream=s)),
    "down_gemv": (1, lambda s: ffn.down_gemv(ga, ua, nv(K, N), stream=s)),
    "fp8_forward": (2, lambda s: ffn.fp8_forward(x, f8(N, K), f8(N, K), f8(K, N), stream=s)),
    "fp8_dual_gemv": (2, lambda s: ffn.fp8_dual_gemv(x, f8(N, K), f8(N, K), stream=s)),
    "fp8_down_gemv": (1, lambda s: ffn.fp8_down_gemv(ga, ua, f8(K, N), stream=s)),
    "w4a4_dual_gemm": (3, lambda s: ffn.w4a4_dual_gemm(x, mx(N, K), mx(N, K), stream=s)),
    "w4a4_forward": (2, lambda s: ffn.w4a4_forward(x, mx(N, K), mx(N, K), nv(K, N), stream=s)),
    "w4a4_down_gemm": (2, lambda s: ffn.w4a4_down_gemm(At((0, N), BF), mx(K, N), stream=s)),
    "w4a4_forward_fp4": (2, lambda s: ffn.w4a4_forward_fp4(x, mx(N, K), mx(N, K), mx(K, N), stream=s)),
    "int8_rmsnorm": (3, lambda s: ffn.int8_rmsnorm(x, At((K,), BF), residual=x, stream=s)),
    "int8_quantize": (2, lambda s: ffn.int8_quantize(x, stream=s)),
    "int8_gemm": (1, lambda s: ffn.int8_gemm(xq, xs, i8(N, K), stream=s)),
    "int8_dual_gemm": (3, lambda s: ffn.int8_dual_gemm(xq, xs, i8(N, K), i8(N, K), stream=s)),
    "int8_forward": (2, lambda s: ffn.int8_forward(xq, xs, i8(N, K), i8(N, K), i8(K, N), stream=s)),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_calls_stream(name, monkeypatch):
    count, call = CALLS[name]
    current, side = Stream(1), Stream(2)
    active, made = [current], []

    @contextlib.contextmanager
    def on(s):
        active.append(s)
        yield
        active.pop()

    def empty(shape, dtype=None, device=None):
        if device is None:
            return torch.zeros(shape, dtype=dtype)
        t = At(shape if isinstance(shape, tuple) else (shape,), dtype, device)
        t.stream, t.recorded = active[-1], []
        made.append(t)
        return t

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[-1])
    call(side)
    assert len(made) == count
    assert all(t.stream is side and t.recorded == [current] for t in made)
    made.clear()
    call(current)
    assert len(made) == count
    assert all(t.stream is current and not t.recorded for t in made)


@pytest.mark.gpu
def test_freed_memory_of_the_current_stream_is_not_taken():
    """A tensor dropped while the current stream has yet to read it, then a call on another stream whose result has its
    size: the result is elsewhere, and the read finds what was there."""
    side = torch.cuda.Stream()
    w = torch.randn(4096, 4096, device="cuda").to(BF)
    torch.cuda.synchronize()
    for _ in range(3):
        old = torch.full((4096, 4096), 3, dtype=I8, device="cuda")
        at = old.data_ptr()
        torch.cuda._sleep(20_000_000)
        total = old.double().sum()
        del old
        codes, scales = ffn.int8_quantize(w, stream=side)
        assert codes.data_ptr() != at
        torch.cuda.current_stream().wait_stream(side)
        again = ffn.int8_quantize(w)
        assert float(total) == 3.0 * 4096 * 4096
        assert torch.equal(codes, again[0]) and torch.equal(scales, again[1])
        del codes, scales


def test_quantize_weight_reads_scale2_on_the_calls_stream(monkeypatch):
    """The read back to the host waits for the stream that writes scale2, not for the current one."""
    current, side = Stream(1), Stream(2)
    active, seen = [current], []

    @contextlib.contextmanager
    def on(s):
        active.append(s)
        yield
        active.pop()

    class Scale:
        def cpu(self):
            seen.append(active[-1])
            return [0.5]

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[-1])
    monkeypatch.setattr(ffn, "quantize", lambda w, stream=None: ("codes", "scales", Scale()))
    for s in (side, None):
        assert ffn.quantize_weight(None, stream=s).scale2 == 0.5
    assert seen == [side, current]


@pytest.mark.gpu
def test_quantize_weight_on_a_busy_stream():
    w = (torch.randn(1024, 2048, device="cuda") * 0.02).to(BF)
    ref = ffn.quantize_weight(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = ffn.quantize_weight(w, stream=side)
        assert got.scale2 == ref.scale2
        assert torch.equal(got.codes, ref.codes) and torch.equal(got.scales, ref.scales)
