"""Host-only checks of the sparse FFN's operators (no GPU): exports, status codes and workspace sizes of the C ABI, and
the binding's argument checks. Every call fails validation or is an empty call, so no HIP work is enqueued; fake
device addresses are never touched."""
import ctypes

import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn
from test_binding_host import Fake

A = 0x7F0000000000  # 16-byte aligned, never dereferenced


def W(codes=A, scales=A, scale2=A):
    return ctypes.byref(ffn.MoeWeightStruct(codes, scales, scale2))


def route(l=A, T=1, E=16, dt=0, b=None, k=2, score=0, norm=1, scale=1.0, ids=A, w=A):
    return ffn.load().ffn_moe_route(l, T, E, dt, b, k, score, norm, scale, ids, w, 0)


def plan(ids=A, T=1, k=2, E=16, rows=A, offsets=A, places=A, ws=A, wsb=1 << 30):
    return ffn.load().ffn_moe_plan(ids, T, k, E, rows, offsets, places, ws, wsb, 0)


def gemm(x=A, xr=4, dt=0, rows=None, k=1, offsets=A, R=4, E=16, K=256, N=512, w=None, odt=0, out=A):
    return ffn.load().ffn_moe_gemm(x, xr, dt, rows, k, offsets, R, E, K, N, w or W(), odt, out, 0)


def fwd(x=A, T=1, K=256, N=512, E=16, k=2, dt=0, ids=A, p=A, g=None, u=None, d=None, act=0, ws=A, wsb=1 << 40, out=A):
    return ffn.load().ffn_moe_forward(x, T, K, N, E, k, dt, ids, p, g or W(), u or W(), d or W(), act, ws, wsb, out, 0)


def test_exports():
    names = ffn.header_functions(ffn.MOE_HEADER_PATH)
    assert set(names) == {"ffn_moe_route", "ffn_moe_plan", "ffn_moe_plan_workspace_bytes", "ffn_moe_gemm",
                          "ffn_moe_forward", "ffn_moe_workspace_bytes"}
    for n in names:
        assert hasattr(ffn.load(), n), n


def test_null():
    assert route(l=None) == route(ids=None) == route(w=None) == ffn.ERR_NULL
    assert plan(ids=None) == plan(rows=None) == plan(offsets=None) == plan(places=None) == ffn.ERR_NULL
    assert plan(T=65536, k=8, ws=None) == ffn.ERR_NULL
    assert gemm(x=None) == gemm(offsets=None) == gemm(out=None) == ffn.ERR_NULL
    for bad in (W(None), W(A, None), W(A, A, None)):
        assert gemm(w=bad) == fwd(g=bad) == fwd(u=bad) == fwd(d=bad) == ffn.ERR_NULL
    assert fwd(x=None) == fwd(ids=None) == fwd(p=None) == fwd(ws=None) == fwd(out=None) == ffn.ERR_NULL
    assert ffn.load().ffn_moe_gemm(A, 4, 0, None, 1, A, 4, 16, 256, 512, None, 0, A, 0) == ffn.ERR_NULL


def test_alignment():
    assert route(l=A + 8) == route(b=A + 2) == route(ids=A + 2) == route(w=A + 1) == ffn.ERR_ALIGN
    assert plan(ids=A + 2) == plan(rows=A + 2) == plan(offsets=A + 1) == plan(places=A + 2) == plan(ws=A + 8) == ffn.ERR_ALIGN
    assert gemm(x=A + 8) == gemm(rows=A + 2, k=2) == gemm(offsets=A + 2) == gemm(out=A + 4) == ffn.ERR_ALIGN
    for bad in (W(A + 8), W(A, A + 1), W(A, A, A + 2)):
        assert gemm(w=bad) == fwd(g=bad) == fwd(u=bad) == fwd(d=bad) == ffn.ERR_ALIGN
    assert fwd(x=A + 2) == fwd(ids=A + 2) == fwd(p=A + 1) == fwd(ws=A + 8) == fwd(out=A + 8) == ffn.ERR_ALIGN


@pytest.mark.parametrize("bad", [0, -32, 16, 48, 65568])
def test_shapes(bad):
    assert gemm(K=bad) == fwd(K=bad) == fwd(N=bad) == ffn.ERR_SHAPE
    assert ffn.moe_workspace_bytes(1, 2, 16, bad, 512) == ffn.moe_workspace_bytes(1, 2, 16, 512, bad) == 0


def test_experts_channels_and_batches():
    for E in (0, -1, 1025):
        assert route(E=E) == plan(E=E) == gemm(E=E) == fwd(E=E) == ffn.ERR_SHAPE
        assert ffn.moe_workspace_bytes(1, 2, E, 256, 512) == ffn.moe_plan_workspace_bytes(65536, 2, E) == 0
    for N in (0, -1, (1 << 20) + 1):
        assert gemm(N=N) == ffn.ERR_SHAPE
    for T in (-1, 65537):
        assert route(T=T) == plan(T=T) == fwd(T=T) == ffn.ERR_BATCH
        assert ffn.moe_workspace_bytes(T, 2, 16, 256, 512) == ffn.moe_plan_workspace_bytes(T, 2, 16) == 0
    for k in (0, -1, 33):
        assert route(k=k, E=64) == plan(k=k) == fwd(k=k) == gemm(rows=A, k=k) == ffn.ERR_BATCH
    assert route(k=17, E=16) == ffn.ERR_BATCH  # more than there are
    assert gemm(R=-1) == gemm(R=65536 * 32 + 1, xr=65536 * 32) == gemm(xr=-1) == ffn.ERR_BATCH
    assert gemm(R=5, xr=4) == ffn.ERR_BATCH  # rows of x that are not there
    assert gemm(k=2) == ffn.ERR_BATCH        # a divisor without rows
    assert gemm(rows=A, k=2, xr=0) == ffn.ERR_BATCH


def test_types_and_values():
    assert route(dt=3) == route(dt=-1) == route(score=2) == route(score=-1) == ffn.ERR_ACT
    assert gemm(dt=2, odt=2) == gemm(dt=-1) == gemm(dt=0, odt=1) == gemm(dt=1, odt=0) == gemm(odt=3) == ffn.ERR_ACT
    assert fwd(dt=2) == fwd(act=2) == fwd(act=-1) == ffn.ERR_ACT
    for v in (float("nan"), float("inf")):
        assert route(scale=v) == ffn.ERR_SCALE2


def test_workspace():
    need = ffn.moe_workspace_bytes(3, 2, 16, 256, 512)
    assert need >= 6 * (4 * 256 + 2 * 512)
    assert fwd(T=3, wsb=need - 1) == ffn.ERR_WORKSPACE
    need = ffn.moe_plan_workspace_bytes(65536, 8, 256)
    assert need > 0 and plan(T=65536, k=8, E=256, wsb=need - 1) == ffn.ERR_WORKSPACE
    assert ffn.moe_plan_workspace_bytes(1, 8, 256) == 0 and ffn.moe_workspace_bytes(0, 2, 16, 256, 512) == 0


def test_empty_calls():
    """No tokens: the rest is validated and nothing launched, whatever the pointers. (A plan of no tokens writes its
    offsets, so it is not among these.)"""
    assert route(T=0, l=None, ids=None, w=None) == ffn.OK
    assert gemm(R=0, xr=0, x=None, offsets=None, out=None) == ffn.OK
    assert fwd(T=0, x=None, ids=None, p=None, ws=None, out=None) == ffn.OK
    assert gemm(R=0, xr=0, w=W(None)) == fwd(T=0, d=W(None)) == ffn.ERR_NULL


# -------------------------------------------------------------------- binding

T, E, k, K, N, R = 3, 8, 2, 256, 512, 6
BF, I, F, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


def we(rows, cols, experts=E, **kw):
    return ffn.MoeDeviceWeight(Fake((experts, rows, cols // 2), **kw), Fake((experts, rows, cols // 16), **kw),
                               Fake((experts,), F, **kw))


@pytest.mark.parametrize("kw", [
    dict(x=Fake((T, K), F)), dict(x=Fake((T, K), BF, contiguous=False)), dict(x=Fake((T, K), BF, device="cpu")),
    dict(ids=Fake((T, k), torch.int64)), dict(ids=Fake((T + 1, k), I)), dict(ids=Fake((T, k), I, contiguous=False)),
    dict(weights=Fake((T, k + 1), F)), dict(weights=Fake((T, k), BF)), dict(gate=we(K, N)), dict(up=we(N, K, E + 1)),
    dict(up=we(N, K, device="cuda:1")), dict(down=we(N, K)), dict(out=Fake((T, K), torch.float16)),
    dict(out=Fake((T, N), BF)), dict(workspace=Fake((1 << 20,), U8, device="cuda:1")),
    dict(workspace=Fake((1 << 20,), U8, contiguous=False)),
    dict(gate=ffn.MoeDeviceWeight(Fake((E, N, K // 2)), Fake((E, N, K // 32)), Fake((E,), F))),
    dict(gate=ffn.MoeDeviceWeight(Fake((E, N, K // 2)), Fake((E, N, K // 16)), Fake((E,), torch.float64))),
])
def test_forward_binding_refuses(kw):
    a = dict(x=Fake((T, K), BF), ids=Fake((T, k), I), weights=Fake((T, k), F), gate=we(N, K), up=we(N, K),
             down=we(K, N), out=Fake((T, K), BF), workspace=Fake((1 << 20,), U8))
    a.update(kw)
    with pytest.raises(ValueError):
        ffn.moe_forward(a.pop("x"), a.pop("ids"), a.pop("weights"), a.pop("gate"), a.pop("up"), a.pop("down"), **a)


@pytest.mark.parametrize("kw", [
    dict(x=Fake((R, K), F)), dict(x=Fake((R, K + 32), BF)), dict(offsets=Fake((E,), I)),
    dict(offsets=Fake((E + 1,), torch.int64)), dict(rows=Fake((R,), torch.int64)), dict(out=Fake((R, N), torch.float16)),
    dict(out=Fake((R + 1, N), BF)), dict(out_dtype=torch.float16), dict(out_dtype=F),
    dict(w=we(N, K, device="cuda:1")),
])
def test_gemm_binding_refuses(kw):
    class Rows(Fake):
        def numel(self):
            return self.shape[0]
    a = dict(x=Fake((R, K), BF), offsets=Fake((E + 1,), I), w=we(N, K), out=Fake((R, N), BF))
    a.update(kw)
    if "rows" in a:
        a["rows"] = Rows(a["rows"].shape, a["rows"].dtype)
    with pytest.raises(ValueError):
        ffn.moe_gemm(a.pop("x"), a.pop("offsets"), a.pop("w"), **a)


@pytest.mark.parametrize("kw", [
    dict(logits=Fake((T, E), torch.int32)), dict(logits=Fake((T, E), BF, contiguous=False)), dict(bias=Fake((E,), BF)),
    dict(bias=Fake((E + 1,), F)), dict(ids=Fake((T, k), torch.int64)), dict(weights=Fake((T, k + 1), F)),
    dict(bias=Fake((E,), F, device="cuda:1")),
])
def test_route_binding_refuses(kw):
    a = dict(logits=Fake((T, E), BF), ids=Fake((T, k), I), weights=Fake((T, k), F))
    a.update(kw)
    with pytest.raises(ValueError):
        ffn.moe_route(a.pop("logits"), k, **a)


@pytest.mark.parametrize("kw", [
    dict(ids=Fake((T, k), torch.int64)), dict(rows=Fake((T, k), I)), dict(offsets=Fake((E,), I)),
    dict(places=Fake((T * k,), I)), dict(workspace=Fake((8,), U8, device="cuda:1")),
])
def test_plan_binding_refuses(kw):
    a = dict(ids=Fake((T, k), I), rows=Fake((T * k,), I), offsets=Fake((E + 1,), I), places=Fake((T, k), I))
    a.update(kw)
    with pytest.raises(ValueError):
        ffn.moe_plan(a.pop("ids"), E, **a)


def test_another_device_is_refused(monkeypatch):
    """The library launches on the current device, so tensors of another one are refused, a stream given or not."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        ffn.moe_route(Fake((T, E), BF), k, ids=Fake((T, k), I), weights=Fake((T, k), F), stream=5)
    with pytest.raises(ValueError, match="current device"):
        ffn.moe_gemm(Fake((R, K), BF), Fake((E + 1,), I), we(N, K), out=Fake((R, N), BF))
