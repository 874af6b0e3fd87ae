"""Buffers of the sparse FFN's operators that overlap are refused (no GPU: no call gets as far as a launch; fake device
addresses are never touched)."""
import ctypes

import pytest

import w4a16_nvfp4_dense_amd as ffn

T, E, K, N, k = 8, 16, 256, 512, 2
R = T * k
STEP = 1 << 32  # further apart than any buffer is long
NEAR = 64       # bytes: aligned, inside every buffer but the scale2's
NAMES = ["x", "logits", "bias", "ids", "weights", "rows", "offsets", "places", "ws", "out", "gc", "gs", "g2", "uc", "us", "u2",
         "dc", "ds", "d2"]
AT = {n: 0x7F0000000000 + i * STEP for i, n in enumerate(NAMES)}


def places(kw):
    return {**AT, **kw}


def weight(a, p):
    return ctypes.byref(ffn.MoeWeightStruct(a[p + "c"], a[p + "s"], a[p + "2"]))


def route(**kw):
    a = places(kw)
    return ffn.load().ffn_moe_route(a["logits"], T, E, 2, a["bias"], k, 0, 1, 1.0, a["ids"], a["weights"], 0)


def plan(tokens=T, **kw):
    a = places(kw)
    return ffn.load().ffn_moe_plan(a["ids"], tokens, k, E, a["rows"], a["offsets"], a["places"], a["ws"], 1 << 30, 0)


def gemm(gather=True, out_dtype=0, **kw):
    a = places(kw)
    return ffn.load().ffn_moe_gemm(a["x"], T if gather else R, 0, a["rows"] if gather else None, k if gather else 1,
                                   a["offsets"], R, E, K, N, weight(a, "g"), out_dtype, a["out"], 0)


def forward(**kw):
    a = places(kw)
    need = ffn.moe_workspace_bytes(T, k, E, K, N)
    return ffn.load().ffn_moe_forward(a["x"], T, K, N, E, k, 0, a["ids"], a["weights"], weight(a, "g"), weight(a, "u"),
                                      weight(a, "d"), 0, a["ws"], need, a["out"], 0)


BYTES = dict(x=T * K * 2, logits=T * E * 4, bias=E * 4, ids=R * 4, weights=R * 4, rows=R * 4, offsets=(E + 1) * 4,
             places=R * 4, out=T * K * 2, gc=E * N * K // 2, gs=E * N * K // 16, g2=E * 4)
for p in "ud":
    BYTES.update({p + "c": BYTES["gc"], p + "s": BYTES["gs"], p + "2": BYTES["g2"]})


def overlapping(written, others):
    """Each written buffer at another's place, a little into it, and at its last aligned piece."""
    for w in written:
        for o in others:
            if o != w:
                last = (BYTES[o] - 1) // 16 * 16 if o in BYTES else 0
                for at in {0, min(NEAR, last), last}:
                    yield pytest.param({w: AT[o] + at}, id=f"{w}-{o}-{at}")


@pytest.mark.parametrize("kw", overlapping(["ids", "weights"], ["logits", "bias", "ids", "weights"]))
def test_route(kw):
    assert route(**kw) == ffn.ERR_ALIAS


@pytest.mark.parametrize("kw", overlapping(["rows", "offsets", "places"], ["ids", "rows", "offsets", "places"]))
def test_plan(kw):
    assert plan(**kw) == ffn.ERR_ALIAS


@pytest.mark.parametrize("other", ["ids", "rows", "offsets", "places"])
def test_plan_workspace(other):
    assert ffn.moe_plan_workspace_bytes(65536, k, E) > 0
    assert plan(tokens=65536, ws=AT[other]) == plan(tokens=65536, **{other: AT["ws"] + NEAR}) == ffn.ERR_ALIAS


@pytest.mark.parametrize("kw", overlapping(["out"], ["x", "rows", "offsets", "gc", "gs", "g2"]))
@pytest.mark.parametrize("out_dtype", [0, 2])
def test_gemm(kw, out_dtype):
    assert gemm(out_dtype=out_dtype, **kw) == ffn.ERR_ALIAS
    if AT["rows"] <= kw["out"] < AT["rows"] + STEP:
        return  # (without them there is no such buffer)
    assert gemm(gather=False, out_dtype=out_dtype, **kw) == ffn.ERR_ALIAS


def test_gemm_an_input_behind_the_first_row_of_out():
    for name in ("x", "rows", "offsets", "gc", "gs", "g2"):
        assert gemm(**{name: AT["out"] + R * N * 2 - 16}) == gemm(out_dtype=2, **{name: AT["out"] + R * N * 4 - 16}) == ffn.ERR_ALIAS


FORWARD = ["x", "ids", "weights", *(p + m for p in "gud" for m in "cs2")]


@pytest.mark.parametrize("kw", [c for c in overlapping(["ws", "out"], [*FORWARD, "ws", "out"]) if c.id != "out-x-0"])
def test_forward(kw):
    assert forward(**kw) == ffn.ERR_ALIAS


@pytest.mark.parametrize("other", [*FORWARD, "out"])
def test_forward_workspace_to_its_last_byte(other):
    need = ffn.moe_workspace_bytes(T, k, E, K, N)
    assert forward(**{other: AT["ws"] + need - 16}) == ffn.ERR_ALIAS
