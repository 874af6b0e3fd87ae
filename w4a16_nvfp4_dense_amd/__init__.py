"""Python binding of libffn_nvfp4 (MI355X / gfx950 NVFP4 W4A16 gated FFN).

Argument marshalling only: every step of the FFN runs in the HIP kernels of
``lib/libffn_nvfp4.so`` through its C ABI (``include/ffn_nvfp4.h``). PyTorch
is used for device memory and streams. There is no fallback: if the library
is missing or a call fails, an exception is raised.

The functions mirror the C entry points:

* :func:`forward`    -- ``ffn_nvfp4_forward``   out = W_d (act(W_g x) * (W_u x))
* :func:`forward_noalloc` -- ``ffn_nvfp4_forward_noalloc`` the same with the
  library's static scratch instead of a workspace (allocates nothing)
* :func:`dual_gemv`  -- ``ffn_nvfp4_dual_gemv`` gate, up = W_g x, W_u x (fp32)
* :func:`down_gemv`  -- ``ffn_nvfp4_down_gemv`` out = W_d bf16(act(gate) * up)
* :func:`workspace_bytes` -- ``ffn_nvfp4_workspace_bytes``
* :func:`quantize`   -- ``ffn_nvfp4_quantize``  bf16 weight -> NVFP4 codes, scales, scale2
* :func:`quantize_workspace_bytes` -- ``ffn_nvfp4_quantize_workspace_bytes``

and, for block-scaled FP8 weights (``include/ffn_fp8.h``):

* :func:`fp8_forward`    -- ``ffn_fp8_forward``
* :func:`fp8_dual_gemv`  -- ``ffn_fp8_dual_gemv``
* :func:`fp8_down_gemv`  -- ``ffn_fp8_down_gemv``
* :func:`fp8_workspace_bytes` -- ``ffn_fp8_workspace_bytes``

the streaming-read ceiling the decode GEMVs are measured against
(``include/ffn_diag.h``):

* :func:`diag_read` -- ``ffn_diag_read`` one launch reading device buffers once

and the W4A4 prefill arm over MXFP4 operands (``include/ffn_w4a4.h``):

* :func:`w4a4_prepare_weight` -- ``ffn_w4a4_prepare_weight`` NVFP4 -> MXFP4 (once)
* :func:`w4a4_dual_gemm`  -- ``ffn_w4a4_dual_gemm``
* :func:`w4a4_forward`    -- ``ffn_w4a4_forward``
* :func:`w4a4_workspace_bytes` -- ``ffn_w4a4_workspace_bytes``
* :func:`w4a4_down_gemm`  -- ``ffn_w4a4_down_gemm`` (the down projection on 4 bits)
* :func:`w4a4_forward_fp4` -- ``ffn_w4a4_forward_fp4`` (all three projections on 4 bits)
* :func:`w4a4_fp4_workspace_bytes` -- ``ffn_w4a4_fp4_workspace_bytes``

and the int8 (W8A8) arm with the operators around it (``include/ffn_int8.h``):

* :func:`int8_rmsnorm`   -- ``ffn_int8_rmsnorm`` norm of x + residual -> int8 codes, scales
* :func:`int8_quantize`  -- ``ffn_int8_quantize`` rows -> int8 codes, scales
* :func:`int8_quantize_weight` -- the same as an :class:`Int8DeviceWeight`
* :func:`int8_prepare_weight`  -- ``ffn_int8_prepare_weight`` NVFP4 -> int8 (once)
* :func:`int8_gemm`      -- ``ffn_int8_gemm`` the product with token and channel scales
* :func:`int8_dual_gemm` -- ``ffn_int8_dual_gemm`` act(gate) * up -> int8 codes, scales
* :func:`int8_forward`   -- ``ffn_int8_forward`` the whole FFN
* :func:`int8_gemm_workspace_bytes`, :func:`int8_workspace_bytes`

and the sparse (mixture of experts) FFN over NVFP4 experts (``include/ffn_moe.h``):

* :func:`moe_route`   -- ``ffn_moe_route`` the top_k experts of each token and their weights
* :func:`moe_plan`    -- ``ffn_moe_plan`` expert order of the chosen (token, expert) pairs
* :func:`moe_gemm`    -- ``ffn_moe_gemm`` the product grouped by expert, ragged sizes
* :func:`moe_forward` -- ``ffn_moe_forward`` the whole sparse FFN
* :func:`moe_plan_workspace_bytes`, :func:`moe_workspace_bytes`
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional, Sequence

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "lib", "libffn_nvfp4.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "ffn_nvfp4.h")
FP8_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "ffn_fp8.h")
W4A4_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "ffn_w4a4.h")
INT8_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "ffn_int8.h")
MOE_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "ffn_moe.h")
DIAG_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "ffn_diag.h")

ACT_SILU = 0
ACT_GELU_TANH = 1

SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1

OK = 0
ERR_NULL = -1
ERR_ALIGN = -2
ERR_SHAPE = -3
ERR_BATCH = -4
ERR_ACT = -5
ERR_WORKSPACE = -6
ERR_LAUNCH = -7
ERR_SCALE2 = -8
ERR_ALIAS = -9


class FfnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({strerror(status)})")


class WeightStruct(ctypes.Structure):
    """ffn_nvfp4_weight: device codes, device scales, host fp32 scale2."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("scale2", ctypes.c_float)]


class Fp8WeightStruct(ctypes.Structure):
    """ffn_fp8_weight: device codes, device fp32 block-scale grid."""

    _fields_ = [("codes", ctypes.c_void_p), ("block_scale", ctypes.c_void_p)]


class MxWeightStruct(ctypes.Structure):
    """ffn_mxfp4_weight: device codes, device E8M0 bytes, host fp32 scale2."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("scale2", ctypes.c_float)]


class Int8WeightStruct(ctypes.Structure):
    """ffn_int8_weight: device codes, device fp32 scale for each row."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class MoeWeightStruct(ctypes.Structure):
    """ffn_moe_weight: device codes, scales and fp32 scale2 of E experts."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("scale2", ctypes.c_void_p)]


_lib: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_WP = ctypes.POINTER(WeightStruct)
_FP = ctypes.POINTER(Fp8WeightStruct)
_MP = ctypes.POINTER(MxWeightStruct)
_QP = ctypes.POINTER(Int8WeightStruct)
_EP = ctypes.POINTER(MoeWeightStruct)


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m w4a16_nvfp4_dense_amd.build` "
                           "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(path)
    lib.ffn_nvfp4_version.restype = _I
    lib.ffn_nvfp4_version.argtypes = []
    lib.ffn_nvfp4_strerror.restype = ctypes.c_char_p
    lib.ffn_nvfp4_strerror.argtypes = [_I]
    lib.ffn_nvfp4_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_nvfp4_workspace_bytes.argtypes = [_I, _I, _I]
    lib.ffn_nvfp4_forward.restype = _I
    lib.ffn_nvfp4_forward.argtypes = [_P, _I, _I, _I, _WP, _WP, _WP, _I, _P, ctypes.c_size_t, _P, _P]
    lib.ffn_nvfp4_forward_noalloc.restype = _I
    lib.ffn_nvfp4_forward_noalloc.argtypes = [_P, _I, _I, _I, _WP, _WP, _WP, _I, _P, _P]
    lib.ffn_nvfp4_dual_gemv.restype = _I
    lib.ffn_nvfp4_dual_gemv.argtypes = [_P, _I, _I, _I, _WP, _WP, _P, _P, _P]
    lib.ffn_nvfp4_down_gemv.restype = _I
    lib.ffn_nvfp4_down_gemv.argtypes = [_P, _P, _I, _I, _I, _WP, _I, _P, _P]
    lib.ffn_nvfp4_quantize_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_nvfp4_quantize_workspace_bytes.argtypes = [_I, _I]
    lib.ffn_nvfp4_quantize.restype = _I
    lib.ffn_nvfp4_quantize.argtypes = [_P, _I, _I, _P, _P, _P, _P, ctypes.c_size_t, _P]
    lib.ffn_fp8_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_fp8_workspace_bytes.argtypes = [_I, _I, _I]
    lib.ffn_fp8_forward.restype = _I
    lib.ffn_fp8_forward.argtypes = [_P, _I, _I, _I, _FP, _FP, _FP, _I, _P, ctypes.c_size_t, _P, _P]
    lib.ffn_fp8_dual_gemv.restype = _I
    lib.ffn_fp8_dual_gemv.argtypes = [_P, _I, _I, _I, _FP, _FP, _P, _P, _P]
    lib.ffn_fp8_down_gemv.restype = _I
    lib.ffn_fp8_down_gemv.argtypes = [_P, _P, _I, _I, _I, _FP, _I, _P, _P]
    lib.ffn_w4a4_prepare_weight.restype = _I
    lib.ffn_w4a4_prepare_weight.argtypes = [_WP, _I, _I, _P, _P, _P]
    lib.ffn_w4a4_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_w4a4_workspace_bytes.argtypes = [_I, _I, _I]
    lib.ffn_w4a4_dual_gemm.restype = _I
    lib.ffn_w4a4_dual_gemm.argtypes = [_P, _I, _I, _I, _MP, _MP, _P, _P, _P, ctypes.c_size_t, _P]
    lib.ffn_diag_read.restype = _I
    lib.ffn_diag_read.argtypes = [ctypes.POINTER(_P), ctypes.POINTER(ctypes.c_size_t), _I, _P, _P]
    lib.ffn_w4a4_forward.restype = _I
    lib.ffn_w4a4_forward.argtypes = [_P, _I, _I, _I, _MP, _MP, _WP, _I, _P, ctypes.c_size_t, _P, _P]
    lib.ffn_w4a4_fp4_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_w4a4_fp4_workspace_bytes.argtypes = [_I, _I, _I]
    lib.ffn_w4a4_down_gemm.restype = _I
    lib.ffn_w4a4_down_gemm.argtypes = [_P, _I, _I, _I, _MP, _P, _P, ctypes.c_size_t, _P]
    lib.ffn_w4a4_forward_fp4.restype = _I
    lib.ffn_w4a4_forward_fp4.argtypes = [_P, _I, _I, _I, _MP, _MP, _MP, _I, _P, ctypes.c_size_t, _P, _P]
    lib.ffn_int8_rmsnorm.restype = _I
    lib.ffn_int8_rmsnorm.argtypes = [_P, _P, _P, _I, _I, _I, _I, ctypes.c_float, ctypes.c_float, _P, _P, _P, _P, _P]
    lib.ffn_int8_quantize.restype = _I
    lib.ffn_int8_quantize.argtypes = [_P, _I, _I, _I, _P, _P, _P]
    lib.ffn_int8_prepare_weight.restype = _I
    lib.ffn_int8_prepare_weight.argtypes = [_WP, _I, _I, _P, _P, _P]
    lib.ffn_int8_gemm_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_int8_gemm_workspace_bytes.argtypes = [_I, _I, _I]
    lib.ffn_int8_gemm.restype = _I
    lib.ffn_int8_gemm.argtypes = [_P, _P, _I, _I, _I, _QP, _P, _I, _P, _P, ctypes.c_size_t, _P]
    lib.ffn_int8_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_int8_workspace_bytes.argtypes = [_I, _I, _I]
    lib.ffn_int8_dual_gemm.restype = _I
    lib.ffn_int8_dual_gemm.argtypes = [_P, _P, _I, _I, _I, _QP, _QP, _I, _P, _P, _P, ctypes.c_size_t, _P]
    lib.ffn_int8_forward.restype = _I
    lib.ffn_int8_forward.argtypes = [_P, _P, _I, _I, _I, _QP, _QP, _QP, _I, _I, _P, ctypes.c_size_t, _P, _P]
    lib.ffn_moe_route.restype = _I
    lib.ffn_moe_route.argtypes = [_P, _I, _I, _I, _P, _I, _I, _I, ctypes.c_float, _P, _P, _P]
    lib.ffn_moe_plan_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_moe_plan_workspace_bytes.argtypes = [_I, _I, _I]
    lib.ffn_moe_plan.restype = _I
    lib.ffn_moe_plan.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, ctypes.c_size_t, _P]
    lib.ffn_moe_gemm.restype = _I
    lib.ffn_moe_gemm.argtypes = [_P, _I, _I, _P, _I, _P, _I, _I, _I, _I, _EP, _I, _P, _P]
    lib.ffn_moe_workspace_bytes.restype = ctypes.c_size_t
    lib.ffn_moe_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
    lib.ffn_moe_forward.restype = _I
    lib.ffn_moe_forward.argtypes = [_P, _I, _I, _I, _I, _I, _I, _P, _P, _EP, _EP, _EP, _I, _P, ctypes.c_size_t, _P,
                                    _P]
    _lib = lib
    return lib


def header_functions(path: str = HEADER_PATH) -> Sequence[str]:
    """Names of the functions a public header declares."""
    import re
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(ffn_(?:nvfp4|fp8|w4a4|int8|moe|diag)_[a-z_0-9]+)\s*\(", text)))


def version() -> int:
    return load().ffn_nvfp4_version()


def strerror(status: int) -> str:
    return load().ffn_nvfp4_strerror(int(status)).decode()


def workspace_bytes(M: int, K: int, N: int) -> int:
    return int(load().ffn_nvfp4_workspace_bytes(int(M), int(K), int(N)))


# ------------------------------------------------------------ torch marshalling


@dataclasses.dataclass
class DeviceWeight:
    """An NVFP4 weight resident on the GPU: codes uint8 [rows, cols/2],
    scales uint8 [rows, cols/16] (both torch tensors on the device) and the
    per-tensor scale2 (host float)."""

    codes: "object"
    scales: "object"
    scale2: float

    @property
    def rows(self) -> int:
        return int(self.codes.shape[0])

    @property
    def cols(self) -> int:
        return int(self.codes.shape[1]) * 2

    def struct(self) -> WeightStruct:
        return WeightStruct(self.codes.data_ptr(), self.scales.data_ptr(), float(self.scale2))

    @classmethod
    def from_host(cls, w, device="cuda") -> "DeviceWeight":
        """From an object with numpy ``codes``, ``scales`` and ``scale2``."""
        import torch
        return cls(torch.from_numpy(w.codes).to(device), torch.from_numpy(w.scales).to(device),
                   float(w.scale2))


def _stream_handle(stream) -> int:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:  # the same handle without building a Stream object
            return raw(torch._C._cuda_getDevice())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _torch_stream(stream):
    """A stream argument (a torch stream or a raw handle) as a torch stream."""
    import torch
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))


def _empty(shape, dtype, device, stream):
    """A tensor for a call on `stream` to write. On a stream other than the
    current one it comes from that stream's pool: memory of the current
    stream's pool may still be in use by what the caller enqueued there before,
    which `stream` does not wait for. It is marked as used on the current
    stream too, so that a caller may go on with it there (having waited for
    `stream`) and drop it."""
    import torch
    if stream is not None:
        s = _torch_stream(stream)
        current = torch.cuda.current_stream()
        if int(s.cuda_stream) != int(current.cuda_stream):
            with torch.cuda.stream(s):
                t = torch.empty(shape, dtype=dtype, device=device)
            t.record_stream(current)
            return t
    return torch.empty(shape, dtype=dtype, device=device)


def _check_tensor(t, dtype, shape, name, device=None):
    dev = t.device
    if (t.dtype == dtype and t.shape == shape and t.is_contiguous()
            and dev.type == "cuda" and (device is None or dev == device)):
        return
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check(status: int, what: str) -> None:
    if status != OK:
        raise FfnError(status, what)


def _check_nvfp4_weight(w: "DeviceWeight", rows: int, cols: int, name: str, device) -> None:
    """An NVFP4 weight of logical shape [rows, cols]: contiguous uint8 codes
    [rows, cols/2] and scales [rows, cols/16] on the device of the call (the C
    ABI sees only pointers, so a mismatched weight would be read out of
    bounds)."""
    import torch
    if cols % 16:
        raise ValueError(f"{name}: {cols} columns is not a multiple of 16")
    _check_tensor(w.codes, torch.uint8, (rows, cols // 2), f"{name}.codes", device)
    _check_tensor(w.scales, torch.uint8, (rows, cols // 16), f"{name}.scales", device)


def forward(x, gate: DeviceWeight, up: DeviceWeight, down: DeviceWeight, act: int = ACT_SILU,
            out=None, workspace=None, stream=None):
    """out[M, K] (bf16) = W_d (act(W_g x) * (W_u x)) for x bf16 [M, K]."""
    import torch
    M, K = x.shape
    N = gate.rows
    _check_tensor(x, torch.bfloat16, (M, K), "x")
    _check_nvfp4_weight(gate, N, K, "gate", x.device)
    _check_nvfp4_weight(up, N, K, "up", x.device)
    _check_nvfp4_weight(down, K, N, "down", x.device)
    if out is None:
        out = _empty((M, K), torch.bfloat16, x.device, stream)
    _check_tensor(out, torch.bfloat16, (M, K), "out", x.device)
    need = workspace_bytes(M, K, N)
    if workspace is None:
        workspace = _empty(max(need, 1), torch.uint8, x.device, stream)
    g, u, d = gate.struct(), up.struct(), down.struct()
    rc = load().ffn_nvfp4_forward(x.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d),
                                  int(act), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_nvfp4_forward")
    return out


def forward_noalloc(x, gate: DeviceWeight, up: DeviceWeight, down: DeviceWeight, out, act: int = ACT_SILU,
                    stream=None):
    """:func:`forward` through ``ffn_nvfp4_forward_noalloc``: the caller
    passes ``out`` (bf16 [M, K]); no device memory is allocated, by the
    library or here."""
    import torch
    M, K = x.shape
    N = gate.rows
    _check_tensor(x, torch.bfloat16, (M, K), "x")
    _check_nvfp4_weight(gate, N, K, "gate", x.device)
    _check_nvfp4_weight(up, N, K, "up", x.device)
    _check_nvfp4_weight(down, K, N, "down", x.device)
    _check_tensor(out, torch.bfloat16, (M, K), "out", x.device)
    g, u, d = gate.struct(), up.struct(), down.struct()
    rc = load().ffn_nvfp4_forward_noalloc(x.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d),
                                          int(act), out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_nvfp4_forward_noalloc")
    return out


def dual_gemv(x, gate: DeviceWeight, up: DeviceWeight, gate_out=None, up_out=None, stream=None):
    """(gate, up) fp32 [M, N] = (scale2_g W_g x, scale2_u W_u x)."""
    import torch
    M, K = x.shape
    N = gate.rows
    _check_tensor(x, torch.bfloat16, (M, K), "x")
    _check_nvfp4_weight(gate, N, K, "gate", x.device)
    _check_nvfp4_weight(up, N, K, "up", x.device)
    if gate_out is None:
        gate_out = _empty((M, N), torch.float32, x.device, stream)
    if up_out is None:
        up_out = _empty((M, N), torch.float32, x.device, stream)
    _check_tensor(gate_out, torch.float32, (M, N), "gate_out", x.device)
    _check_tensor(up_out, torch.float32, (M, N), "up_out", x.device)
    g, u = gate.struct(), up.struct()
    rc = load().ffn_nvfp4_dual_gemv(x.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u),
                                    gate_out.data_ptr(), up_out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_nvfp4_dual_gemv")
    return gate_out, up_out


def down_gemv(gate_in, up_in, down: DeviceWeight, act: int = ACT_SILU, out=None, stream=None):
    """out[M, K] (bf16) = W_d bf16(act(gate) * up) with the activation fused
    into the down GEMV's input load."""
    import torch
    M, N = gate_in.shape
    K = down.rows
    _check_tensor(gate_in, torch.float32, (M, N), "gate_in")
    _check_tensor(up_in, torch.float32, (M, N), "up_in", gate_in.device)
    _check_nvfp4_weight(down, K, N, "down", gate_in.device)
    if out is None:
        out = _empty((M, K), torch.bfloat16, gate_in.device, stream)
    _check_tensor(out, torch.bfloat16, (M, K), "out", gate_in.device)
    d = down.struct()
    rc = load().ffn_nvfp4_down_gemv(gate_in.data_ptr(), up_in.data_ptr(), M, N, K, ctypes.byref(d), int(act),
                                    out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_nvfp4_down_gemv")
    return out


def quantize_workspace_bytes(rows: int, cols: int) -> int:
    return int(load().ffn_nvfp4_quantize_workspace_bytes(int(rows), int(cols)))


def quantize(w, codes=None, scales=None, scale2=None, workspace=None, stream=None):
    """NVFP4 of the bf16 weight w [rows, cols]: (codes uint8 [rows, cols/2],
    scales uint8 [rows, cols/16], scale2 fp32 [1]), all on w's device."""
    import torch
    rows, cols = w.shape
    _check_tensor(w, torch.bfloat16, (rows, cols), "w")
    dev = w.device
    if codes is None:
        codes = _empty((rows, cols // 2), torch.uint8, dev, stream)
    if scales is None:
        scales = _empty((rows, cols // 16), torch.uint8, dev, stream)
    if scale2 is None:
        scale2 = _empty(1, torch.float32, dev, stream)
    _check_tensor(codes, torch.uint8, (rows, cols // 2), "codes", dev)
    _check_tensor(scales, torch.uint8, (rows, cols // 16), "scales", dev)
    _check_tensor(scale2, torch.float32, (1,), "scale2", dev)
    need = quantize_workspace_bytes(rows, cols)
    if workspace is None:
        workspace = _empty(max(need, 4), torch.uint8, dev, stream)
    rc = load().ffn_nvfp4_quantize(w.data_ptr(), rows, cols, codes.data_ptr(), scales.data_ptr(),
                                   scale2.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(rc, "ffn_nvfp4_quantize")
    return codes, scales, scale2


def quantize_weight(w, stream=None) -> DeviceWeight:
    """:func:`quantize` as a DeviceWeight (waits for the result, on the call's
    stream, to read scale2 back to the host)."""
    import torch
    codes, scales, scale2 = quantize(w, stream=stream)
    if stream is None:
        value = scale2.cpu()
    else:
        with torch.cuda.stream(_torch_stream(stream)):
            value = scale2.cpu()
    return DeviceWeight(codes, scales, float(value[0]))


def bf16_from_bits(bits, device="cuda"):
    """A bf16 torch tensor on ``device`` from a numpy uint16 array of bf16 bits."""
    import numpy as np
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits, dtype=np.uint16).view(np.int16))
    return t.view(torch.bfloat16).to(device)


def bf16_to_f64(t):
    """A bf16 torch tensor as a float64 numpy array (exact)."""
    return t.float().cpu().double().numpy()


# ------------------------------------------------------------ FP8 weights


@dataclasses.dataclass
class Fp8DeviceWeight:
    """A block-scaled FP8 weight resident on the GPU: codes uint8 [rows, cols]
    (E4M3FN bytes) and block_scale float32 [ceil(rows/128), ceil(cols/128)]."""

    codes: "object"
    block_scale: "object"

    @property
    def rows(self) -> int:
        return int(self.codes.shape[0])

    @property
    def cols(self) -> int:
        return int(self.codes.shape[1])

    def struct(self) -> Fp8WeightStruct:
        return Fp8WeightStruct(self.codes.data_ptr(), self.block_scale.data_ptr())

    @classmethod
    def from_host(cls, w, device="cuda") -> "Fp8DeviceWeight":
        """From an object with numpy ``codes`` and ``block_scale``."""
        import torch
        return cls(torch.from_numpy(w.codes).to(device), torch.from_numpy(w.block_scale).to(device))


def _check_fp8_weight(w: Fp8DeviceWeight, rows: int, cols: int, name: str, device=None) -> None:
    import torch
    _check_tensor(w.codes, torch.uint8, (rows, cols), f"{name}.codes", device)
    _check_tensor(w.block_scale, torch.float32, ((rows + 127) // 128, (cols + 127) // 128), f"{name}.block_scale",
                  device)


def fp8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(load().ffn_fp8_workspace_bytes(int(M), int(K), int(N)))


def fp8_forward(x, gate: Fp8DeviceWeight, up: Fp8DeviceWeight, down: Fp8DeviceWeight, act: int = ACT_SILU,
                out=None, workspace=None, stream=None):
    """out[M, K] (bf16) = W_d (act(W_g x) * (W_u x)) over FP8 weights."""
    import torch
    M, K = x.shape
    N = gate.rows
    _check_tensor(x, torch.bfloat16, (M, K), "x")
    _check_fp8_weight(gate, N, K, "gate", x.device)
    _check_fp8_weight(up, N, K, "up", x.device)
    _check_fp8_weight(down, K, N, "down", x.device)
    if out is None:
        out = _empty((M, K), torch.bfloat16, x.device, stream)
    _check_tensor(out, torch.bfloat16, (M, K), "out", x.device)
    need = fp8_workspace_bytes(M, K, N)
    if workspace is None:
        workspace = _empty(max(need, 1), torch.uint8, x.device, stream)
    g, u, d = gate.struct(), up.struct(), down.struct()
    rc = load().ffn_fp8_forward(x.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d),
                                int(act), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_fp8_forward")
    return out


def fp8_dual_gemv(x, gate: Fp8DeviceWeight, up: Fp8DeviceWeight, gate_out=None, up_out=None, stream=None):
    """(gate, up) fp32 [M, N] = (W_g x, W_u x) over FP8 weights."""
    import torch
    M, K = x.shape
    N = gate.rows
    _check_tensor(x, torch.bfloat16, (M, K), "x")
    _check_fp8_weight(gate, N, K, "gate", x.device)
    _check_fp8_weight(up, N, K, "up", x.device)
    if gate_out is None:
        gate_out = _empty((M, N), torch.float32, x.device, stream)
    if up_out is None:
        up_out = _empty((M, N), torch.float32, x.device, stream)
    _check_tensor(gate_out, torch.float32, (M, N), "gate_out", x.device)
    _check_tensor(up_out, torch.float32, (M, N), "up_out", x.device)
    g, u = gate.struct(), up.struct()
    rc = load().ffn_fp8_dual_gemv(x.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u),
                                  gate_out.data_ptr(), up_out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_fp8_dual_gemv")
    return gate_out, up_out


def fp8_down_gemv(gate_in, up_in, down: Fp8DeviceWeight, act: int = ACT_SILU, out=None, stream=None):
    """out[M, K] (bf16) = W_d bf16(act(gate) * up) over an FP8 W_d, with the
    activation fused into the down GEMV's input load."""
    import torch
    M, N = gate_in.shape
    K = down.rows
    _check_tensor(gate_in, torch.float32, (M, N), "gate_in")
    _check_tensor(up_in, torch.float32, (M, N), "up_in", gate_in.device)
    _check_fp8_weight(down, K, N, "down", gate_in.device)
    if out is None:
        out = _empty((M, K), torch.bfloat16, gate_in.device, stream)
    _check_tensor(out, torch.bfloat16, (M, K), "out", gate_in.device)
    d = down.struct()
    rc = load().ffn_fp8_down_gemv(gate_in.data_ptr(), up_in.data_ptr(), M, N, K, ctypes.byref(d), int(act),
                                  out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_fp8_down_gemv")
    return out


# ------------------------------------------------------------ W4A4 (MXFP4)


@dataclasses.dataclass
class MxDeviceWeight:
    """An MXFP4 weight on the GPU: codes uint8 [rows, cols/2], E8M0 scales
    uint8 [rows, cols/32], and the host fp32 scale2."""

    codes: "object"
    scales: "object"
    scale2: float

    @property
    def rows(self) -> int:
        return int(self.codes.shape[0])

    @property
    def cols(self) -> int:
        return int(self.codes.shape[1]) * 2

    def struct(self) -> MxWeightStruct:
        return MxWeightStruct(self.codes.data_ptr(), self.scales.data_ptr(), float(self.scale2))


def _check_mx_weight(w: MxDeviceWeight, rows: int, cols: int, name: str, device) -> None:
    """An MXFP4 weight of logical shape [rows, cols]: contiguous uint8 codes
    [rows, cols/2] and E8M0 bytes [rows, cols/32] on the device of the call."""
    import torch
    if cols % 32:
        raise ValueError(f"{name}: {cols} columns is not a multiple of 32")
    _check_tensor(w.codes, torch.uint8, (rows, cols // 2), f"{name}.codes", device)
    _check_tensor(w.scales, torch.uint8, (rows, cols // 32), f"{name}.scales", device)


def w4a4_prepare_weight(w: DeviceWeight, stream=None) -> MxDeviceWeight:
    """Requantise an NVFP4 weight to MXFP4 on the GPU (asynchronous)."""
    import torch
    rows, cols = w.rows, w.cols
    dev = w.codes.device
    _check_nvfp4_weight(w, rows, cols, "w", dev)
    codes = _empty((rows, cols // 2), torch.uint8, dev, stream)
    scales = _empty((rows, cols // 32), torch.uint8, dev, stream)
    st = w.struct()
    rc = load().ffn_w4a4_prepare_weight(ctypes.byref(st), rows, cols, codes.data_ptr(), scales.data_ptr(),
                                        _stream_handle(stream))
    _check(rc, "ffn_w4a4_prepare_weight")
    return MxDeviceWeight(codes, scales, float(w.scale2))


def w4a4_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(load().ffn_w4a4_workspace_bytes(int(M), int(K), int(N)))


def w4a4_dual_gemm(x, gate: MxDeviceWeight, up: MxDeviceWeight, gate_out=None, up_out=None, workspace=None,
                   stream=None):
    """(gate, up) fp32 [M, N] over MXFP4 activations and weights."""
    import torch
    M, K = x.shape
    N = gate.rows
    _check_tensor(x, torch.bfloat16, (M, K), "x")
    _check_mx_weight(gate, N, K, "gate", x.device)
    _check_mx_weight(up, N, K, "up", x.device)
    if gate_out is None:
        gate_out = _empty((M, N), torch.float32, x.device, stream)
    if up_out is None:
        up_out = _empty((M, N), torch.float32, x.device, stream)
    _check_tensor(gate_out, torch.float32, (M, N), "gate_out", x.device)
    _check_tensor(up_out, torch.float32, (M, N), "up_out", x.device)
    if workspace is None:
        workspace = _empty(max(w4a4_workspace_bytes(M, K, N), 1), torch.uint8, x.device, stream)
    g, u = gate.struct(), up.struct()
    rc = load().ffn_w4a4_dual_gemm(x.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u), gate_out.data_ptr(),
                                   up_out.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(rc, "ffn_w4a4_dual_gemm")
    return gate_out, up_out


def w4a4_forward(x, gate: MxDeviceWeight, up: MxDeviceWeight, down: DeviceWeight, act: int = ACT_SILU, out=None,
                 workspace=None, stream=None):
    """out[M, K] (bf16): W4A4 gate and up, then the NVFP4 down projection."""
    import torch
    M, K = x.shape
    N = gate.rows
    _check_tensor(x, torch.bfloat16, (M, K), "x")
    _check_mx_weight(gate, N, K, "gate", x.device)
    _check_mx_weight(up, N, K, "up", x.device)
    _check_nvfp4_weight(down, K, N, "down", x.device)
    if out is None:
        out = _empty((M, K), torch.bfloat16, x.device, stream)
    _check_tensor(out, torch.bfloat16, (M, K), "out", x.device)
    if workspace is None:
        workspace = _empty(max(w4a4_workspace_bytes(M, K, N), 1), torch.uint8, x.device, stream)
    g, u, d = gate.struct(), up.struct(), down.struct()
    rc = load().ffn_w4a4_forward(x.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), int(act),
                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(), out.data_ptr(),
                                 _stream_handle(stream))
    _check(rc, "ffn_w4a4_forward")
    return out


def w4a4_fp4_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(load().ffn_w4a4_fp4_workspace_bytes(int(M), int(K), int(N)))


def w4a4_down_gemm(h, down: MxDeviceWeight, out=None, workspace=None, stream=None):
    """out[M, K] (bf16) = scale2 * (mx(h) . mx(W_d)) for h [M, N] bf16 and an
    MXFP4 down weight [K, N]."""
    import torch
    M, N = h.shape
    K = down.rows
    _check_tensor(h, torch.bfloat16, (M, N), "h")
    _check_mx_weight(down, K, N, "down", h.device)
    if out is None:
        out = _empty((M, K), torch.bfloat16, h.device, stream)
    _check_tensor(out, torch.bfloat16, (M, K), "out", h.device)
    if workspace is None:
        workspace = _empty(max(w4a4_fp4_workspace_bytes(M, K, N), 1), torch.uint8, h.device, stream)
    d = down.struct()
    rc = load().ffn_w4a4_down_gemm(h.data_ptr(), M, N, K, ctypes.byref(d), out.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(rc, "ffn_w4a4_down_gemm")
    return out


def w4a4_forward_fp4(x, gate: MxDeviceWeight, up: MxDeviceWeight, down: MxDeviceWeight, act: int = ACT_SILU,
                     out=None, workspace=None, stream=None):
    """out[M, K] (bf16): all three projections on 4 bits (MXFP4 weights and
    activations, h quantised before the down projection)."""
    import torch
    M, K = x.shape
    N = gate.rows
    _check_tensor(x, torch.bfloat16, (M, K), "x")
    _check_mx_weight(gate, N, K, "gate", x.device)
    _check_mx_weight(up, N, K, "up", x.device)
    _check_mx_weight(down, K, N, "down", x.device)
    if out is None:
        out = _empty((M, K), torch.bfloat16, x.device, stream)
    _check_tensor(out, torch.bfloat16, (M, K), "out", x.device)
    if workspace is None:
        workspace = _empty(max(w4a4_fp4_workspace_bytes(M, K, N), 1), torch.uint8, x.device, stream)
    g, u, d = gate.struct(), up.struct(), down.struct()
    rc = load().ffn_w4a4_forward_fp4(x.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d),
                                     int(act), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_w4a4_forward_fp4")
    return out


# ------------------------------------------------------------ int8 (W8A8)


@dataclasses.dataclass
class Int8DeviceWeight:
    """An int8 weight on the GPU: codes int8 [rows, cols] and one fp32 scale
    for each row (output channel) [rows]."""

    codes: "object"
    scales: "object"

    @property
    def rows(self) -> int:
        return int(self.codes.shape[0])

    @property
    def cols(self) -> int:
        return int(self.codes.shape[1])

    def struct(self) -> Int8WeightStruct:
        return Int8WeightStruct(self.codes.data_ptr(), self.scales.data_ptr())

    @classmethod
    def from_host(cls, w, device="cuda") -> "Int8DeviceWeight":
        """From an object with numpy ``codes`` and ``scales``."""
        import torch
        return cls(torch.from_numpy(w.codes).to(device), torch.from_numpy(w.scales).to(device))


_INT8_DTYPES: dict = {}  # torch type -> ffn_int8_dtype, filled at first use


def _int8_dtype(dtype, name: str) -> int:
    """ffn_int8_dtype of a torch type."""
    if not _INT8_DTYPES:
        import torch
        _INT8_DTYPES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    code = _INT8_DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {dtype}")
    return code


def _check_int8_weight(w: Int8DeviceWeight, rows: int, cols: int, name: str, device) -> None:
    """An int8 weight of logical shape [rows, cols] on the device of the call."""
    import torch
    c, s = w.codes, w.scales
    if (c.dtype == torch.int8 and c.shape == (rows, cols) and c.is_contiguous() and c.device == device
            and s.dtype == torch.float32 and s.shape == (rows,) and s.is_contiguous() and s.device == device):
        return
    _check_tensor(w.codes, torch.int8, (rows, cols), f"{name}.codes", device)
    _check_tensor(w.scales, torch.float32, (rows,), f"{name}.scales", device)


def _check_workspace(workspace, device) -> None:
    if workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def int8_rmsnorm(x, weight, eps: float = 1e-6, residual=None, weight_offset: float = 0.0, codes=None, scales=None,
                 sum_out=None, y_out=None, stream=None):
    """(codes int8 [M, K], scales fp32 [M], t) of the root-mean-square norm of
    t = x + residual: the int8 rows of t / sqrt(mean t^2 + eps) *
    (weight_offset + weight). t (x's type, the new residual stream) is None
    without a residual, unless ``sum_out`` is given; ``sum_out`` may be x or
    residual. ``y_out`` (x's type), if given, receives the norm itself, for
    arms that take real activations."""
    import torch
    M, K = x.shape
    dtype, wdtype = _int8_dtype(x.dtype, "x"), _int8_dtype(weight.dtype, "weight")
    dev = x.device
    _check_tensor(x, x.dtype, (M, K), "x")
    _check_tensor(weight, weight.dtype, (K,), "weight", dev)
    if residual is not None:
        _check_tensor(residual, x.dtype, (M, K), "residual", dev)
    if codes is None:
        codes = _empty((M, K), torch.int8, dev, stream)
    else:
        _check_tensor(codes, torch.int8, (M, K), "codes", dev)
    if scales is None:
        scales = _empty(M, torch.float32, dev, stream)
    else:
        _check_tensor(scales, torch.float32, (M,), "scales", dev)
    if sum_out is None:
        if residual is not None:
            sum_out = _empty((M, K), x.dtype, dev, stream)
    else:
        _check_tensor(sum_out, x.dtype, (M, K), "sum_out", dev)
    if y_out is not None:
        _check_tensor(y_out, x.dtype, (M, K), "y_out", dev)
    rc = load().ffn_int8_rmsnorm(x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(),
                                 M, K, dtype, wdtype, eps, weight_offset, codes.data_ptr(), scales.data_ptr(),
                                 None if sum_out is None else sum_out.data_ptr(),
                                 None if y_out is None else y_out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_int8_rmsnorm")
    return codes, scales, sum_out


def int8_quantize(x, codes=None, scales=None, stream=None):
    """(codes int8 [rows, cols], scales fp32 [rows]) of the rows of x."""
    import torch
    rows, cols = x.shape
    dtype = _int8_dtype(x.dtype, "x")
    dev = x.device
    _check_tensor(x, x.dtype, (rows, cols), "x")
    if codes is None:
        codes = _empty((rows, cols), torch.int8, dev, stream)
    else:
        _check_tensor(codes, torch.int8, (rows, cols), "codes", dev)
    if scales is None:
        scales = _empty(rows, torch.float32, dev, stream)
    else:
        _check_tensor(scales, torch.float32, (rows,), "scales", dev)
    rc = load().ffn_int8_quantize(x.data_ptr(), rows, cols, dtype, codes.data_ptr(), scales.data_ptr(),
                                  _stream_handle(stream))
    _check(rc, "ffn_int8_quantize")
    return codes, scales


def int8_quantize_weight(w, stream=None) -> Int8DeviceWeight:
    """:func:`int8_quantize` of a weight [N, K] as an Int8DeviceWeight (asynchronous)."""
    return Int8DeviceWeight(*int8_quantize(w, stream=stream))


def int8_prepare_weight(w: DeviceWeight, stream=None) -> Int8DeviceWeight:
    """An NVFP4 weight as int8 rows on the GPU (asynchronous)."""
    import torch
    rows, cols = w.rows, w.cols
    dev = w.codes.device
    _check_nvfp4_weight(w, rows, cols, "w", dev)
    codes = _empty((rows, cols), torch.int8, dev, stream)
    scales = _empty(rows, torch.float32, dev, stream)
    st = w.struct()
    rc = load().ffn_int8_prepare_weight(ctypes.byref(st), rows, cols, codes.data_ptr(), scales.data_ptr(),
                                        _stream_handle(stream))
    _check(rc, "ffn_int8_prepare_weight")
    return Int8DeviceWeight(codes, scales)


def int8_gemm_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(load().ffn_int8_gemm_workspace_bytes(int(M), int(K), int(N)))


def int8_gemm(xq, xs, w: Int8DeviceWeight, bias=None, out_dtype=None, out=None, workspace=None, stream=None):
    """out[M, N] = xs * w.scales * (xq . w.codes) + bias in ``out_dtype`` (the
    type of ``out`` if that is given, else bfloat16); xq int8 [M, K], xs fp32 [M]."""
    import torch
    M, K = xq.shape
    N = w.rows
    dev = xq.device
    _check_tensor(xq, torch.int8, (M, K), "xq")
    _check_tensor(xs, torch.float32, (M,), "xs", dev)
    _check_int8_weight(w, N, K, "w", dev)
    if bias is not None:
        _check_tensor(bias, torch.float32, (N,), "bias", dev)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    dtype = _int8_dtype(out_dtype, "out")
    if out is None:
        out = _empty((M, N), out_dtype, dev, stream)
    else:
        _check_tensor(out, out_dtype, (M, N), "out", dev)
    lib = load()
    need = lib.ffn_int8_gemm_workspace_bytes(M, K, N)
    if workspace is None:
        if need:
            workspace = _empty(need, torch.uint8, dev, stream)
    else:
        _check_workspace(workspace, dev)
    st = w.struct()
    rc = lib.ffn_int8_gemm(xq.data_ptr(), xs.data_ptr(), M, K, N, ctypes.byref(st),
                           None if bias is None else bias.data_ptr(), dtype, out.data_ptr(),
                           None if workspace is None else workspace.data_ptr(),
                           0 if workspace is None else workspace.numel() * workspace.element_size(),
                           _stream_handle(stream))
    _check(rc, "ffn_int8_gemm")
    return out


def int8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(load().ffn_int8_workspace_bytes(int(M), int(K), int(N)))


def int8_dual_gemm(xq, xs, gate: Int8DeviceWeight, up: Int8DeviceWeight, act: int = ACT_SILU, hq=None, hs=None,
                   workspace=None, stream=None):
    """(hq int8 [M, N], hs fp32 [M]): the int8 rows of act(W_g x) * (W_u x)."""
    import torch
    M, K = xq.shape
    N = gate.rows
    dev = xq.device
    _check_tensor(xq, torch.int8, (M, K), "xq")
    _check_tensor(xs, torch.float32, (M,), "xs", dev)
    _check_int8_weight(gate, N, K, "gate", dev)
    _check_int8_weight(up, N, K, "up", dev)
    if hq is None:
        hq = _empty((M, N), torch.int8, dev, stream)
    else:
        _check_tensor(hq, torch.int8, (M, N), "hq", dev)
    if hs is None:
        hs = _empty(M, torch.float32, dev, stream)
    else:
        _check_tensor(hs, torch.float32, (M,), "hs", dev)
    lib = load()
    need = lib.ffn_int8_workspace_bytes(M, K, N)
    if workspace is None:
        workspace = _empty(max(need, 1), torch.uint8, dev, stream)
    else:
        _check_workspace(workspace, dev)
    g, u = gate.struct(), up.struct()
    rc = lib.ffn_int8_dual_gemm(xq.data_ptr(), xs.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u), int(act),
                                hq.data_ptr(), hs.data_ptr(), workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(rc, "ffn_int8_dual_gemm")
    return hq, hs


def int8_forward(xq, xs, gate: Int8DeviceWeight, up: Int8DeviceWeight, down: Int8DeviceWeight, act: int = ACT_SILU,
                 out_dtype=None, out=None, workspace=None, stream=None):
    """out[M, K] = W_d q(act(W_g x) * (W_u x)) over int8 weights, for x as
    int8 rows (xq int8 [M, K], xs fp32 [M]); ``out_dtype`` as :func:`int8_gemm`."""
    import torch
    M, K = xq.shape
    N = gate.rows
    dev = xq.device
    _check_tensor(xq, torch.int8, (M, K), "xq")
    _check_tensor(xs, torch.float32, (M,), "xs", dev)
    _check_int8_weight(gate, N, K, "gate", dev)
    _check_int8_weight(up, N, K, "up", dev)
    _check_int8_weight(down, K, N, "down", dev)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    dtype = _int8_dtype(out_dtype, "out")
    if out is None:
        out = _empty((M, K), out_dtype, dev, stream)
    else:
        _check_tensor(out, out_dtype, (M, K), "out", dev)
    lib = load()
    need = lib.ffn_int8_workspace_bytes(M, K, N)
    if workspace is None:
        workspace = _empty(max(need, 1), torch.uint8, dev, stream)
    else:
        _check_workspace(workspace, dev)
    g, u, d = gate.struct(), up.struct(), down.struct()
    rc = lib.ffn_int8_forward(xq.data_ptr(), xs.data_ptr(), M, K, N, ctypes.byref(g), ctypes.byref(u),
                              ctypes.byref(d), int(act), dtype, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_int8_forward")
    return out


# ------------------------------------------------------------ sparse FFN (mixture of experts)


@dataclasses.dataclass
class MoeDeviceWeight:
    """NVFP4 weights of E experts on the GPU: codes uint8 [E, rows, cols/2],
    scales uint8 [E, rows, cols/16], scale2 float32 [E]."""

    codes: "object"
    scales: "object"
    scale2: "object"

    @property
    def experts(self) -> int:
        return int(self.codes.shape[0])

    @property
    def rows(self) -> int:
        return int(self.codes.shape[1])

    @property
    def cols(self) -> int:
        return int(self.codes.shape[2]) * 2

    def struct(self) -> MoeWeightStruct:
        return MoeWeightStruct(self.codes.data_ptr(), self.scales.data_ptr(), self.scale2.data_ptr())

    @classmethod
    def stack(cls, weights: Sequence[DeviceWeight]) -> "MoeDeviceWeight":
        """From one :class:`DeviceWeight` for each expert (copies them)."""
        import torch
        dev = weights[0].codes.device
        return cls(torch.stack([w.codes for w in weights]), torch.stack([w.scales for w in weights]),
                   torch.tensor([w.scale2 for w in weights], dtype=torch.float32, device=dev))


def _check_moe_weight(w: MoeDeviceWeight, experts: int, rows: int, cols: int, name: str, device) -> None:
    """NVFP4 weights of logical shape [experts, rows, cols] on the device of the call."""
    import torch
    c, s, s2 = w.codes, w.scales, w.scale2
    if cols % 16:
        raise ValueError(f"{name}: {cols} columns is not a multiple of 16")
    if (c.dtype == torch.uint8 and c.shape == (experts, rows, cols // 2) and c.is_contiguous() and c.device == device
            and s.dtype == torch.uint8 and s.shape == (experts, rows, cols // 16) and s.is_contiguous()
            and s.device == device and s2.dtype == torch.float32 and s2.shape == (experts,) and s2.is_contiguous()
            and s2.device == device):
        return
    _check_tensor(c, torch.uint8, (experts, rows, cols // 2), f"{name}.codes", device)
    _check_tensor(s, torch.uint8, (experts, rows, cols // 16), f"{name}.scales", device)
    _check_tensor(s2, torch.float32, (experts,), f"{name}.scale2", device)


def _check_current(device) -> None:
    """The library launches on the current device, which has to be the tensors'."""
    import torch
    current = torch.cuda.current_device()
    if device.index != current:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{current}")


def _moe_half(dtype, name: str) -> int:
    """ffn_moe_dtype of a 16-bit torch type."""
    code = _int8_dtype(dtype, name)
    if code > 1:
        raise ValueError(f"{name} must be bfloat16 or float16, got {dtype}")
    return code


def moe_route(logits, top_k: int, score: int = SCORE_SOFTMAX, bias=None, normalize: bool = True, scale: float = 1.0,
              ids=None, weights=None, stream=None):
    """(ids int32 [T, top_k], weights fp32 [T, top_k]): the experts of the
    largest keys of each row of ``logits`` [T, E], the largest first, ties to
    the lower expert, and their weights ``scale * score`` (``normalize``: over
    the sum of the chosen scores). The key is the logit, or with ``bias`` (fp32
    [E]) score + bias. Experts with a logit or key of -infinity are not
    chosen: an id of -1 with weight 0 stands where too few are left. Weights
    hold where scores are out of range too; the sigmoid of the type's lowest
    finite value, a mask's, counts as 0."""
    import torch
    T, E = logits.shape
    dev = logits.device
    dtype = _int8_dtype(logits.dtype, "logits")
    _check_tensor(logits, logits.dtype, (T, E), "logits")
    if bias is not None:
        _check_tensor(bias, torch.float32, (E,), "bias", dev)
    if ids is None:
        ids = _empty((T, top_k), torch.int32, dev, stream)
    else:
        _check_tensor(ids, torch.int32, (T, top_k), "ids", dev)
    if weights is None:
        weights = _empty((T, top_k), torch.float32, dev, stream)
    else:
        _check_tensor(weights, torch.float32, (T, top_k), "weights", dev)
    _check_current(dev)
    rc = load().ffn_moe_route(logits.data_ptr(), T, E, dtype, None if bias is None else bias.data_ptr(), top_k,
                              int(score), bool(normalize), scale, ids.data_ptr(), weights.data_ptr(),
                              _stream_handle(stream))
    _check(rc, "ffn_moe_route")
    return ids, weights


def moe_plan_workspace_bytes(T: int, top_k: int, experts: int) -> int:
    return int(load().ffn_moe_plan_workspace_bytes(int(T), int(top_k), int(experts)))


def moe_plan(ids, experts: int, rows=None, offsets=None, places=None, workspace=None, stream=None):
    """(rows int32 [T * top_k], offsets int32 [experts + 1], places int32 [T,
    top_k]): the slots t * top_k + j of ``ids`` int32 [T, top_k] in expert order
    (-1 behind the last expert's), where each expert begins, and the place of
    each slot (-1: its id is no expert)."""
    import torch
    T, top_k = ids.shape
    dev = ids.device
    _check_tensor(ids, torch.int32, (T, top_k), "ids")
    if rows is None:
        rows = _empty((T * top_k,), torch.int32, dev, stream)
    else:
        _check_tensor(rows, torch.int32, (T * top_k,), "rows", dev)
    if offsets is None:
        offsets = _empty((experts + 1,), torch.int32, dev, stream)
    else:
        _check_tensor(offsets, torch.int32, (experts + 1,), "offsets", dev)
    if places is None:
        places = _empty((T, top_k), torch.int32, dev, stream)
    else:
        _check_tensor(places, torch.int32, (T, top_k), "places", dev)
    lib = load()
    if workspace is None:
        need = lib.ffn_moe_plan_workspace_bytes(T, top_k, experts)
        if need:
            workspace = _empty((need,), torch.uint8, dev, stream)
    else:
        _check_workspace(workspace, dev)
    _check_current(dev)
    rc = lib.ffn_moe_plan(ids.data_ptr(), T, top_k, experts, rows.data_ptr(), offsets.data_ptr(), places.data_ptr(),
                          None if workspace is None else workspace.data_ptr(),
                          0 if workspace is None else workspace.numel() * workspace.element_size(),
                          _stream_handle(stream))
    _check(rc, "ffn_moe_plan")
    return rows, offsets, places


def moe_gemm(x, offsets, w: MoeDeviceWeight, rows=None, top_k: int = 1, out_dtype=None, out=None, stream=None):
    """out[i] = w.scale2[e] * W_e x[i] for offsets[e] <= i < offsets[e + 1]
    (``offsets`` int32 [E + 1], ascending, on the device); with ``rows`` int32
    [R], slots of ``top_k`` for each row of x, out[i] is of x[rows[i] // top_k].
    ``out_dtype``: x's type (the default) or float32. Rows of ``out`` outside
    all experts are left as they were."""
    import torch
    x_rows, K = x.shape
    E, N = w.experts, w.rows
    dev = x.device
    dtype = _moe_half(x.dtype, "x")
    _check_tensor(x, x.dtype, (x_rows, K), "x")
    _check_tensor(offsets, torch.int32, (E + 1,), "offsets", dev)
    _check_moe_weight(w, E, N, K, "w", dev)
    R = x_rows
    if rows is not None:
        R = rows.numel()
        _check_tensor(rows, torch.int32, (R,), "rows", dev)
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    if out_dtype != x.dtype and out_dtype != torch.float32:
        raise ValueError(f"out must be {x.dtype} or float32, got {out_dtype}")
    if out is None:
        out = _empty((R, N), out_dtype, dev, stream)
    else:
        _check_tensor(out, out_dtype, (R, N), "out", dev)
    _check_current(dev)
    st = w.struct()
    rc = load().ffn_moe_gemm(x.data_ptr(), x_rows, dtype, None if rows is None else rows.data_ptr(), top_k,
                             offsets.data_ptr(), R, E, K, N, ctypes.byref(st), 2 if out_dtype == torch.float32 else dtype,
                             out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_moe_gemm")
    return out


def moe_workspace_bytes(T: int, top_k: int, experts: int, K: int, N: int) -> int:
    return int(load().ffn_moe_workspace_bytes(int(T), int(top_k), int(experts), int(K), int(N)))


def moe_forward(x, ids, weights, gate: MoeDeviceWeight, up: MoeDeviceWeight, down: MoeDeviceWeight,
                act: int = ACT_SILU, out=None, workspace=None, stream=None):
    """out[t] = sum_j weights[t, j] * W_d,e (act(W_g,e x[t]) * (W_u,e x[t])),
    e = ids[t, j], for x [T, K] (bfloat16 or float16), ids int32 and weights fp32
    [T, top_k]; an id outside 0 .. E - 1 adds nothing. ``out`` may be x."""
    import torch
    T, K = x.shape
    top_k = ids.shape[1]
    E, N = gate.experts, gate.rows
    dev = x.device
    dtype = _moe_half(x.dtype, "x")
    _check_tensor(x, x.dtype, (T, K), "x")
    _check_tensor(ids, torch.int32, (T, top_k), "ids", dev)
    _check_tensor(weights, torch.float32, (T, top_k), "weights", dev)
    _check_moe_weight(gate, E, N, K, "gate", dev)
    _check_moe_weight(up, E, N, K, "up", dev)
    _check_moe_weight(down, E, K, N, "down", dev)
    if out is None:
        out = _empty((T, K), x.dtype, dev, stream)
    else:
        _check_tensor(out, x.dtype, (T, K), "out", dev)
    lib = load()
    if workspace is None:
        workspace = _empty((max(lib.ffn_moe_workspace_bytes(T, top_k, E, K, N), 1),), torch.uint8, dev, stream)
    else:
        _check_workspace(workspace, dev)
    _check_current(dev)
    g, u, d = gate.struct(), up.struct(), down.struct()
    rc = lib.ffn_moe_forward(x.data_ptr(), T, K, N, E, top_k, dtype, ids.data_ptr(), weights.data_ptr(),
                             ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), int(act), workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), out.data_ptr(), _stream_handle(stream))
    _check(rc, "ffn_moe_forward")
    return out


# ------------------------------------------------------------ measurement aid


class DiagRead:
    """Prepared arguments of ``ffn_diag_read`` over a list of device tensors
    (contiguous, sizes multiples of 16 bytes): ``launch(stream)`` enqueues one
    read of all of them."""

    def __init__(self, tensors):
        import torch
        if not 1 <= len(tensors) <= 8:
            raise ValueError("1 to 8 buffers")
        for t in tensors:
            if t.device.type != "cuda" or not t.is_contiguous():
                raise ValueError("buffers must be contiguous GPU tensors")
        self._keep = list(tensors)
        self.n = len(tensors)
        self.bytes = sum(t.numel() * t.element_size() for t in tensors)
        self._ptrs = (_P * self.n)(*[t.data_ptr() for t in tensors])
        self._sizes = (ctypes.c_size_t * self.n)(*[t.numel() * t.element_size() for t in tensors])
        self._sink = torch.zeros(1, dtype=torch.int32, device=tensors[0].device)

    def launch(self, stream=None) -> None:
        rc = load().ffn_diag_read(self._ptrs, self._sizes, self.n, self._sink.data_ptr(), _stream_handle(stream))
        _check(rc, "ffn_diag_read")


def diag_read(tensors, stream=None) -> None:
    """One streaming read of every byte of ``tensors`` (see ``ffn_diag.h``)."""
    DiagRead(tensors).launch(stream)
