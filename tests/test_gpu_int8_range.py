"""The int8 norm over the whole range of fp32 (needs an MI355X): rows whose squares do not fit fp32, too large or
too small, beside ordinary rows. The tolerances are those of test_gpu_int8.py's norm: a row is at most scaled by a
power of two first, which is exact."""
import numpy as np
import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn
from test_gpu_int8 import check_norm, norm64, np_of, rounded, same_bits

pytestmark = pytest.mark.gpu

LARGEST = {"bf16": 3.3e38, "f16": 6.0e4, "f32": 3.3e38}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [16, 1040, 5120, 40000])
def test_large_rows(K, dtype):
    """Largest magnitudes from where a sum of squares just overflows to the type's own, with and without a residual
    (of the other half of the sum, so that t itself stays finite)."""
    rng = np.random.default_rng(K)
    amax = np.array([1.0, 1e17, 1e18, 2e19, 1e25, 1e38, LARGEST[dtype], 3.0])
    v = rng.uniform(-1, 1, (len(amax), K))
    v *= (amax / np.abs(v).max(1))[:, None]
    x = rounded(v, dtype)
    w = rounded(1 + 0.2 * rng.standard_normal(K), "f32")
    codes, scales, _ = ffn.int8_rmsnorm(x.cuda(), w.cuda(), 1e-6)
    _, y = norm64(x, None, w, 1e-6, 0.0)
    check_norm(codes, scales, y)
    half = rounded(np_of(x) / 2, dtype)
    codes, scales, total = ffn.int8_rmsnorm(half.cuda(), w.cuda(), 1e-6, residual=half.cuda())
    t, y = norm64(half, half, w, 1e-6, 0.0)
    check_norm(codes, scales, y)
    assert same_bits(total, rounded((np_of(half) + np_of(half)).astype(np.float32), dtype))
    # the ordinary rows have the bits that they have alone
    c, s, _ = ffn.int8_rmsnorm(half[[0, 7]].cuda(), w.cuda(), 1e-6, residual=half[[0, 7]].cuda())
    assert same_bits(c, codes[[0, 7]]) and same_bits(s, scales[[0, 7]])


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-38, 1e-30, 1e-26])
@pytest.mark.parametrize("K", [16, 5120, 40000])
def test_small_rows(K, eps):
    """Squares that vanish or are subnormal, with an eps of their size or none: down to fp32's smallest numbers."""
    rng = np.random.default_rng(K + 1)
    amax = np.array([1.0, 1e-10, 1e-14, 1e-17, 1e-20, 1e-25, 1e-37, 1e-41, 2.0])
    v = rng.uniform(-1, 1, (len(amax), K))
    v *= (amax / np.abs(v).max(1))[:, None]
    x = rounded(v, "f32")
    w = rounded(1 + 0.2 * rng.standard_normal(K), "f32")
    eps = float(np.float32(eps))
    y_out = torch.empty(x.shape, device="cuda")
    codes, scales, _ = ffn.int8_rmsnorm(x.cuda(), w.cuda(), eps, y_out=y_out)
    _, y = norm64(x, None, w, eps, 0.0)
    keep = np.abs(y).max(1) / 127 >= 2e-38  # (rows below this have scale 0 by the quantiser's rule)
    check_norm(codes[keep], scales[keep], y[keep])
    assert not bool(codes[~keep].any()) and not bool(scales[~keep].any())
    assert np.all(np.abs(np_of(y_out) - y) <= np.abs(y) * (2.0 ** -24 + 4e-6) + 1e-44)


@pytest.mark.parametrize("eps", [1e30, 3e38])
def test_large_eps(eps):
    rng = np.random.default_rng(3)
    x = rounded(rng.standard_normal((4, 512)) * np.array([[1.0], [1e15], [1e19], [1e30]]), "f32")
    w = rounded(np.ones(512), "f32")
    codes, scales, _ = ffn.int8_rmsnorm(x.cuda(), w.cuda(), eps)
    _, y = norm64(x, None, w, float(np.float32(eps)), 0.0)
    check_norm(codes, scales, y)


def test_rows_without_a_norm():
    """Infinities and NaN, in t or only in the sum x + residual: scale NaN, codes 0. So has a row of zeros with
    eps = 0; with an eps it is zeros. The large and the small row between them stand."""
    rng = np.random.default_rng(4)
    v = rng.standard_normal((7, 1024)).astype(np.float32)
    v[0, 5] = np.inf
    v[1] *= np.float32(1e30)
    v[2, 1000] = np.nan
    v[3] *= np.float32(1e-30)
    v[4] = 0
    v[5] = 3e38
    r = np.zeros_like(v)
    r[5] = 3e38
    w = np.ones(1024, np.float32)
    for eps in (0.0, 1e-6):
        x, res = torch.from_numpy(v), torch.from_numpy(r)
        codes, scales, _ = ffn.int8_rmsnorm(x.cuda(), torch.from_numpy(w).cuda(), eps, residual=res.cuda())
        s = scales.cpu().numpy()
        assert np.isnan(s[[0, 2, 5]]).all() and not bool(codes[[0, 2, 4, 5]].any())
        assert np.isnan(s[4]) if eps == 0 else s[4] == 0
        for row in (1, 3, 6):
            _, y = norm64(x[row:row + 1], None, torch.from_numpy(w), float(np.float32(eps)), 0.0)
            check_norm(codes[row:row + 1], scales[row:row + 1], y)
