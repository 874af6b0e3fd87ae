"""Host-only checks of the int8 operators (no GPU): exports, status codes and
workspace sizes of the C ABI, and the binding's argument checks. Every call
fails validation or is an empty call, so no HIP work is enqueued; fake device
addresses are never touched."""
import ctypes

import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn
from test_binding_host import Fake

A = 0x7F0000000000  # 16-byte aligned, never dereferenced
B = A + 0x100000


def W(codes=A, scales=B):
    return ctypes.byref(ffn.Int8WeightStruct(codes, scales))


def norm(x=A, r=A, w=A, M=1, K=256, dt=0, wdt=0, eps=1e-6, off=0.0, q=A, s=A, t=A, y=None):
    return ffn.load().ffn_int8_rmsnorm(x, r, w, M, K, dt, wdt, eps, off, q, s, t, y, 0)


def quant(x=A, rows=1, cols=256, dt=0, q=A, s=A):
    return ffn.load().ffn_int8_quantize(x, rows, cols, dt, q, s, 0)


def gemm(x=A, xs=A, M=1, K=256, N=512, w=None, b=None, dt=0, out=A, ws=None, wsb=0):
    return ffn.load().ffn_int8_gemm(x, xs, M, K, N, w or W(), b, dt, out, ws, wsb, 0)


def dual(x=A, xs=A, M=1, K=256, N=512, g=None, u=None, act=0, hq=A, hs=A, ws=A, wsb=1 << 30):
    return ffn.load().ffn_int8_dual_gemm(x, xs, M, K, N, g or W(), u or W(), act, hq, hs, ws, wsb, 0)


def fwd(x=A, xs=A, M=1, K=256, N=512, g=None, u=None, d=None, act=0, dt=0, ws=A, wsb=1 << 30, out=A):
    return ffn.load().ffn_int8_forward(x, xs, M, K, N, g or W(), u or W(), d or W(), act, dt, ws, wsb, out, 0)


def test_exports():
    names = ffn.header_functions(ffn.INT8_HEADER_PATH)
    assert set(names) == {"ffn_int8_rmsnorm", "ffn_int8_quantize", "ffn_int8_prepare_weight", "ffn_int8_gemm",
                          "ffn_int8_gemm_workspace_bytes", "ffn_int8_dual_gemm", "ffn_int8_forward",
                          "ffn_int8_workspace_bytes"}
    for n in names:
        assert hasattr(ffn.load(), n), n


def test_null():
    assert norm(x=None) == norm(w=None) == norm(q=None) == norm(s=None) == ffn.ERR_NULL
    assert quant(x=None) == quant(q=None) == quant(s=None) == ffn.ERR_NULL
    assert gemm(x=None) == gemm(xs=None) == gemm(out=None) == gemm(w=W(None)) == gemm(w=W(A, None)) == ffn.ERR_NULL
    assert dual(x=None) == dual(xs=None) == dual(hq=None) == dual(hs=None) == dual(ws=None) == ffn.ERR_NULL
    assert fwd(x=None) == fwd(out=None) == fwd(ws=None) == fwd(d=W(None)) == fwd(xs=None) == ffn.ERR_NULL
    lib = ffn.load()
    assert lib.ffn_int8_gemm(A, A, 1, 256, 512, None, None, 0, A, None, 0, 0) == ffn.ERR_NULL
    assert lib.ffn_int8_prepare_weight(None, 16, 32, A, A, 0) == ffn.ERR_NULL


def test_alignment():
    assert norm(x=A + 8) == norm(r=A + 2) == norm(w=A + 4) == norm(q=A + 8) == norm(s=A + 2) == ffn.ERR_ALIGN
    assert norm(t=A + 8) == norm(y=A + 4) == ffn.ERR_ALIGN
    assert quant(x=A + 8) == quant(q=A + 1) == quant(s=A + 1) == ffn.ERR_ALIGN
    assert gemm(x=A + 8) == gemm(xs=A + 2) == gemm(out=A + 4) == gemm(b=A + 2) == gemm(w=W(A + 8)) == ffn.ERR_ALIGN
    assert gemm(w=W(A, A + 2)) == ffn.ERR_ALIGN
    assert dual(hq=A + 8) == dual(hs=A + 1) == dual(ws=A + 8) == dual(u=W(A + 4)) == ffn.ERR_ALIGN
    assert fwd(out=A + 8) == fwd(ws=A + 4) == fwd(x=A + 4) == fwd(g=W(A + 1)) == ffn.ERR_ALIGN


@pytest.mark.parametrize("bad", [0, -16, 8, 40, 65552])
def test_shapes(bad):
    assert norm(K=bad) == quant(cols=bad) == gemm(K=bad) == ffn.ERR_SHAPE
    assert dual(K=bad) == dual(N=bad) == fwd(K=bad) == fwd(N=bad) == ffn.ERR_SHAPE
    assert ffn.int8_workspace_bytes(1, bad, 512) == ffn.int8_workspace_bytes(1, 512, bad) == 0
    assert ffn.int8_gemm_workspace_bytes(1, bad, 512) == 0


def test_channels_and_batches():
    assert gemm(N=0) == gemm(N=-1) == gemm(N=(1 << 20) + 1) == ffn.ERR_SHAPE
    for f in (norm, gemm, dual, fwd):
        assert f(M=-1) == f(M=65537) == ffn.ERR_BATCH
    assert quant(rows=-1) == quant(rows=(1 << 20) + 1) == ffn.ERR_BATCH
    st = ctypes.byref(ffn.WeightStruct(A, B, 1.0))
    lib = ffn.load()
    for rows, cols in ((0, 32), (16, 0), (16, 48), (65537, 32), (16, 65568), (-1, 32)):
        assert lib.ffn_int8_prepare_weight(st, rows, cols, A, A, 0) == ffn.ERR_SHAPE
    assert lib.ffn_int8_prepare_weight(st, 16, 32, A + 8, A, 0) == ffn.ERR_ALIGN
    inf = ctypes.byref(ffn.WeightStruct(A, B, float("inf")))
    assert lib.ffn_int8_prepare_weight(inf, 16, 32, A, A, 0) == ffn.ERR_SCALE2


def test_types_and_values():
    for dt in (-1, 3):
        assert norm(dt=dt) == norm(wdt=dt) == quant(dt=dt) == gemm(dt=dt) == fwd(dt=dt) == ffn.ERR_ACT
    assert dual(act=2) == fwd(act=-1) == ffn.ERR_ACT
    for v in (float("nan"), float("inf"), -1e-6):
        assert norm(eps=v) == ffn.ERR_SCALE2
    assert norm(off=float("nan")) == ffn.ERR_SCALE2


def test_workspace():
    need = ffn.int8_workspace_bytes(3, 256, 512)
    assert need >= 3 * 512 * 5 + 12
    assert dual(M=3, wsb=need - 1) == fwd(M=3, wsb=need - 1) == ffn.ERR_WORKSPACE
    assert ffn.int8_workspace_bytes(0, 256, 512) == 0 and ffn.int8_workspace_bytes(-1, 256, 512) == 0


def test_empty_calls():
    """M = 0 validates the rest and launches nothing, whatever the pointers."""
    assert norm(M=0, x=None, r=None, q=None, s=None, t=None) == ffn.OK
    assert quant(rows=0, x=None, q=None, s=None) == ffn.OK
    assert gemm(M=0, x=None, xs=None, out=None) == ffn.OK
    assert dual(M=0, x=None, xs=None, hq=None, hs=None, ws=None) == ffn.OK
    assert fwd(M=0, x=None, xs=None, ws=None, out=None) == ffn.OK
    assert norm(M=0, w=None) == gemm(M=0, w=W(None)) == fwd(M=0, d=W(None)) == ffn.ERR_NULL


# -------------------------------------------------------------------- binding

M, K, N = 3, 256, 512
I8, F = torch.int8, torch.float32


def w8(rows, cols, **kw):
    return ffn.Int8DeviceWeight(Fake((rows, cols), I8, **kw), Fake((rows,), F, **kw))


def call(**kw):
    a = dict(xq=Fake((M, K), I8), xs=Fake((M,), F), gate=w8(N, K), up=w8(N, K), down=w8(K, N))
    a.update(kw)
    return ffn.int8_forward(a["xq"], a["xs"], a["gate"], a["up"], a["down"], out=a.get("out", Fake((M, K), torch.bfloat16)),
                            workspace=Fake((1 << 20,), torch.uint8), out_dtype=a.get("out_dtype"))


@pytest.mark.parametrize("kw", [
    dict(xq=Fake((M, K), torch.uint8)), dict(xq=Fake((M, K), I8, contiguous=False)), dict(xs=Fake((M + 1,), F)),
    dict(xs=Fake((M,), torch.bfloat16)), dict(gate=w8(K, N)), dict(up=w8(N, K, device="cuda:1")), dict(down=w8(N, K)),
    dict(down=ffn.Int8DeviceWeight(Fake((K, N), I8), Fake((N,), F))), dict(out=Fake((M, N), torch.bfloat16)),
    dict(out=Fake((M, K), torch.float64)), dict(out_dtype=torch.float16), dict(xq=Fake((M, K), I8, device="cpu")),
])
def test_forward_binding_refuses(kw):
    with pytest.raises(ValueError):
        call(**kw)


@pytest.mark.parametrize("kw", [dict(bias=Fake((N + 1,), F)), dict(bias=Fake((N,), torch.bfloat16)),
                                dict(out=Fake((M, K), F)), dict(out_dtype=torch.int32),
                                dict(w=w8(N, K + 16)), dict(xs=Fake((1,), F))])
def test_gemm_binding_refuses(kw):
    a = dict(xs=Fake((M,), F), w=w8(N, K))
    a.update(kw)
    with pytest.raises(ValueError):
        ffn.int8_gemm(Fake((M, K), I8), a["xs"], a["w"], bias=a.get("bias"), out=a.get("out", None if "out_dtype" in a else Fake((M, N), F)),
                      out_dtype=a.get("out_dtype"))


@pytest.mark.parametrize("kw", [dict(weight=Fake((K + 16,), torch.bfloat16)), dict(weight=Fake((K,), torch.float64)),
                                dict(residual=Fake((M, K), F)), dict(residual=Fake((M + 1, K), torch.bfloat16)),
                                dict(codes=Fake((M, K), torch.uint8)), dict(scales=Fake((M, 1), F)),
                                dict(sum_out=Fake((M, K), F)), dict(y_out=Fake((M, K), torch.bfloat16, contiguous=False)),
                                dict(x=Fake((M, K), torch.int8))])
def test_norm_binding_refuses(kw):
    bf = torch.bfloat16
    a = dict(x=Fake((M, K), bf), weight=Fake((K,), bf), residual=Fake((M, K), bf), codes=Fake((M, K), I8),
             scales=Fake((M,), F), sum_out=Fake((M, K), bf), y_out=Fake((M, K), bf))
    a.update(kw)
    with pytest.raises(ValueError):
        ffn.int8_rmsnorm(a.pop("x"), a.pop("weight"), **a)


def test_quantize_and_dual_binding_refuse():
    with pytest.raises(ValueError):
        ffn.int8_quantize(Fake((M, K), torch.float64))
    with pytest.raises(ValueError):
        ffn.int8_quantize(Fake((M, K), F), codes=Fake((M, K), torch.uint8), scales=Fake((M,), F))
    with pytest.raises(ValueError):
        ffn.int8_dual_gemm(Fake((M, K), I8), Fake((M,), F), w8(N, K), w8(K, N), hq=Fake((M, N), I8), hs=Fake((M,), F))
    with pytest.raises(ValueError):
        ffn.int8_prepare_weight(ffn.DeviceWeight(Fake((N, K // 2)), Fake((N, K // 32)), 1.0))
