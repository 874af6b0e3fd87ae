"""Buffers of the int8 norm that overlap in a way it cannot take are refused (no GPU: no call gets as far as a launch;
fake device addresses are never touched)."""
import pytest

import w4a16_nvfp4_dense_amd as ffn

M, K = 4, 256
X, R, W, Q, S, T, Y = (0x7F0000000000 + i * 0x100000 for i in range(7))
NEAR = 64  # bytes: aligned, inside every buffer's first row


def norm(x=X, r=R, w=W, q=Q, s=S, t=T, y=Y, dt=0):
    return ffn.load().ffn_int8_rmsnorm(x, r, w, M, K, dt, 0, 1e-6, 0.0, q, s, t, y, 0)


@pytest.mark.parametrize("kw", [
    dict(y=T), dict(t=X, y=X), dict(t=R, y=R),                                  # both outputs in one place
    dict(y=T + NEAR), dict(t=Y + NEAR),                                         # or partly
    dict(t=X + NEAR), dict(t=R + NEAR), dict(y=X + NEAR), dict(y=R + NEAR),     # an input's place, shifted
    dict(t=X + K * 2), dict(y=R + (M - 1) * K * 2), dict(t=X - 16),             # by a row, to its last row, from before
    dict(q=X), dict(q=R), dict(q=T), dict(q=Y + NEAR), dict(q=W),               # codes in the place of another
    dict(s=Q), dict(s=X), dict(s=T + NEAR), dict(s=W), dict(s=Y),
    dict(t=W), dict(y=W + NEAR),
])
@pytest.mark.parametrize("dt", [0, 2])
def test_refused(kw, dt):
    assert norm(dt=dt, **kw) == ffn.ERR_ALIAS


def test_status_has_a_text():
    assert ffn.ERR_ALIAS == -9 and "overlap" in ffn.strerror(ffn.ERR_ALIAS)
