"""The int8 operators on buffers that the caller brings (needs an MI355X): norms written in the place of their inputs,
the gated product into given codes and scales, and long fp32 rows. Bit for bit against the same calls on fresh
buffers, which the other tests hold against 64 bits, or with their norm's tolerances."""
import numpy as np
import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn
from test_gpu_int8 import _config, check_norm, norm64, np_of, rounded, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (37, 5120), (5, 17408), (300, 1040)])
def test_norm_in_the_place_of_its_inputs(M, K, dtype):
    rng = np.random.default_rng(M + K)
    x, r = (rounded(rng.standard_normal((M, K)), dtype).cuda() for _ in range(2))
    w = rounded(1 + 0.1 * rng.standard_normal(K), dtype).cuda()
    y0 = torch.empty_like(x)
    c0, s0, t0 = ffn.int8_rmsnorm(x, w, residual=r, y_out=y0)
    for t_at, y_at in (("r", "x"), ("x", "r"), (None, "x"), (None, "r"), ("r", None), ("x", None)):
        b = {"x": x.clone(), "r": r.clone()}
        t, y = b.get(t_at), b.get(y_at)
        c, s, total = ffn.int8_rmsnorm(b["x"], w, residual=b["r"], sum_out=t, y_out=y)
        assert same_bits(c, c0) and same_bits(s, s0) and same_bits(total, t0)
        assert t is None or total is t
        assert y is None or same_bits(y, y0)
    b = x.clone()
    y1 = torch.empty_like(x)
    c1, s1, none = ffn.int8_rmsnorm(x, w, y_out=y1)
    c, s, _ = ffn.int8_rmsnorm(b, w, y_out=b)
    assert none is None and same_bits(c, c1) and same_bits(s, s1) and same_bits(b, y1)


def test_norm_of_itself():
    """x given as its own residual: t = 2 x."""
    rng = np.random.default_rng(1)
    x = rounded(rng.standard_normal((9, 656)), "bf16")
    w = rounded(np.ones(656), "bf16")
    c0, s0, t0 = ffn.int8_rmsnorm(x.cuda(), w.cuda(), residual=x.cuda())
    same = x.cuda()
    c, s, t = ffn.int8_rmsnorm(same, w.cuda(), residual=same)
    assert same_bits(c, c0) and same_bits(s, s0) and same_bits(t, t0)
    assert same_bits(t, (2 * x.float()).to(torch.bfloat16))


@pytest.mark.parametrize("K", [32784, 40000, 65536])
@pytest.mark.parametrize("residual", [False, True])
def test_long_fp32_rows(K, residual):
    rng = np.random.default_rng(K)
    x = rounded(rng.standard_normal((3, K)), "f32")
    r = rounded(2 * rng.standard_normal((3, K)), "f32") if residual else None
    w = rounded(0.2 * rng.standard_normal(K), "f32")
    y_out = torch.empty((3, K), device="cuda")
    codes, scales, total = ffn.int8_rmsnorm(x.cuda(), w.cuda(), 1e-6, residual=None if r is None else r.cuda(),
                                            weight_offset=1.0, y_out=y_out)
    _, y = norm64(x, r, w, 1e-6, 1.0)
    check_norm(codes, scales, y)
    # of y_out, with a t rounded to fp32 where it is a sum: |t| 2^-24 more
    t = np_of(x).astype(np.float64) + (0 if r is None else np_of(r).astype(np.float64))
    assert np.all(np.abs(np_of(y_out) - y) <= np.abs(y) * (2.0 ** -23 + 4e-6) + 1e-7)
    if residual:
        assert same_bits(total, rounded(t.astype(np.float32), "f32"))


@pytest.mark.parametrize("M,K,N,act", [(1, 1024, 2048, 0), (3, 272, 1040, 1), (48, 1024, 528, 0), (300, 256, 4112, 1)])
def test_dual_into_given_buffers(M, K, N, act):
    xq, xs, gate, up, _ = _config(M, K, N, M + K + N)
    ref = ffn.int8_dual_gemm(xq, xs, gate, up, act)
    codes = torch.full((M * N + 256,), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((M + 64,), 77.0, device="cuda")
    ws = torch.full((ffn.int8_workspace_bytes(M, K, N) + 256,), 0xEE, dtype=torch.uint8, device="cuda")
    need = ws.numel() - 256
    for _ in range(2):
        hq, hs = ffn.int8_dual_gemm(xq, xs, gate, up, act, hq=codes[:M * N].view(M, N), hs=scales[:M], workspace=ws[:need])
        assert hq.data_ptr() == codes.data_ptr() and hs.data_ptr() == scales.data_ptr()
        assert same_bits(hq, ref[0]) and same_bits(hs, ref[1])
    # nothing behind them is written
    assert bool((codes[M * N:] == 77).all()) and bool((scales[M:] == 77).all()) and bool((ws[need:] == 0xEE).all())


@pytest.mark.parametrize("M,K,N", [(1, 5120, 17408), (24, 4224, 1040), (300, 4112, 4096), (2048, 528, 9232)])
def test_workspaces_hold_what_they_say(M, K, N):
    """The product and the forward write nothing behind their workspaces, at sizes whose tiles are shared."""
    xq, xs, gate, up, down = _config(M, K, N, 3)
    for need, call in ((ffn.int8_gemm_workspace_bytes(M, K, N), lambda ws: ffn.int8_gemm(xq, xs, gate, workspace=ws)),
                       (ffn.int8_workspace_bytes(M, K, N), lambda ws: ffn.int8_forward(xq, xs, gate, up, down, workspace=ws))):
        assert need > 0
        ws = torch.full((need + 65536,), 0x3C, dtype=torch.uint8, device="cuda")
        out = call(ws[:need])
        assert bool((ws[need:] == 0x3C).all())
        assert same_bits(out, call(None))
