"""The router's weights where scores leave the range of 32 and of 64 bits: they are ratios of scores, or scores times a
factor, and hold wherever those are in range."""
import math

import pytest
import torch

import w4a16_nvfp4_dense_amd as ffn
from moe_ref import DEV, U, gen

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def expected(logits, ids, score, normalize, scale):
    """Weights of chosen experts in 64 bits, from logarithms of their scores."""
    l = logits.double()
    log = torch.log_softmax(l, 1) if score == ffn.SCORE_SOFTMAX else torch.nn.functional.logsigmoid(l)
    log = log.gather(1, ids.long())
    return torch.softmax(log, 1) * scale if normalize else torch.exp(log + math.log(scale))


def check(logits, k, score, bias=None, normalize=True, scale=1.0):
    """The kernel's 64-bit arithmetic is off by far less than the rounding to fp32, U; the reference's logarithms, of
    magnitudes up to 2000 and 2^-53 of that, by 2^-42 of the weight. Below 2^-126 a weight's absolute error counts.
    Rows without a bias whose chosen logits are all -80 or more are in 32 bits: a score has an exponential (2 U), a sum
    (U) and a quotient (2 U, not always the nearest), 5 U; the sum of the scores a tree of six levels more, 11 U; their
    quotient 5 + 11 + 2 U, the factor another: 19 U."""
    ids, w = ffn.moe_route(logits, k, score, bias=bias, normalize=normalize, scale=scale)
    key = logits.double() if bias is None else bias.double().expand(logits.shape)  # (the scores are far below the biases)
    assert torch.equal(ids, torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k].int())
    want = expected(logits, ids, score, normalize, scale)
    narrow = (logits.gather(1, ids.long()) >= -80).all(1, keepdim=True) & (bias is None)
    tol = torch.where(narrow, 19 * U, U) + 2.0 ** -40
    assert ((w.double() - want).abs() <= tol * want + 2.0 ** -126).all(), (w, want)


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("E,k", [(3, 3), (8, 2), (64, 8), (160, 6), (300, 32)])
@pytest.mark.parametrize("lo,hi", [(-120, -88), (-90, -86), (-104, -87), (-700, -80), (-1500, -800)])
def test_sigmoid_far_below_zero(dtype, E, k, lo, hi):
    logits = (lo + (hi - lo) * torch.rand(77, E, generator=gen(E - lo), device=DEV)).to(dtype)
    check(logits, k, ffn.SCORE_SIGMOID)
    check(logits, k, ffn.SCORE_SIGMOID, scale=2.5)


@pytest.mark.parametrize("dtype", [BF, HF, F])
def test_sigmoid_two_close_ones(dtype):
    logits = torch.tensor([[-88.0, -89.0], [-95.0, -96.0], [-1000.0, -1001.0]], device=DEV).to(dtype)
    _, w = ffn.moe_route(logits, 2, ffn.SCORE_SIGMOID)
    gap = (logits[:, 0] - logits[:, 1]).double()
    assert ((w[:, 0].double() - 1 / (1 + torch.exp(-gap))).abs() <= U).all()


@pytest.mark.parametrize("dtype", [BF, HF, F])
def test_sigmoid_from_far_below_to_far_above(dtype):
    """Chosen ones of both signs in one row, and of magnitudes whose exponentials are infinite."""
    row = [60000.0, 800.0, 90.0, 3.0, 0.0, -0.5, -40.0, -87.5, -95.0, -800.0, -60000.0]
    logits = torch.tensor([row, row[::-1], [-v for v in row]], device=DEV).to(dtype)
    for k in (1, 4, len(row)):
        check(logits, k, ffn.SCORE_SIGMOID)
        check(logits, k, ffn.SCORE_SIGMOID, normalize=False)
    check(logits[:, 5:].contiguous(), 6, ffn.SCORE_SIGMOID)


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("with_bias", [False, True])
def test_sigmoid_times_a_large_factor(dtype, with_bias):
    """scale * score is in range where the score alone is not (2^100 e^-110 is 2e-18)."""
    logits = (-110 + 30 * torch.rand(50, 40, generator=gen(3), device=DEV)).to(dtype)
    bias = torch.rand(40, generator=gen(4), device=DEV) if with_bias else None
    check(logits, 5, ffn.SCORE_SIGMOID, bias=bias, normalize=False, scale=2.0 ** 100)


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_softmax_times_a_large_factor(dtype, normalize, with_bias):
    """The same of a softmax whose largest logit is far above the others (of 2^100 e^-110 among them)."""
    E, k = 70, 6
    logits = (-110 + 15 * torch.rand(50, E, generator=gen(5), device=DEV)).to(dtype)
    logits[:, 33] = 0
    bias = None
    if with_bias:
        bias = 2 + torch.rand(E, generator=gen(6), device=DEV)
        bias[33] = 9
    ids, w = ffn.moe_route(logits, k, ffn.SCORE_SOFTMAX, bias=bias, normalize=normalize, scale=2.0 ** 100)
    key = logits.double() if bias is None else bias.double().expand(logits.shape)
    assert torch.equal(ids, torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k].int())
    want = expected(logits, ids, ffn.SCORE_SOFTMAX, normalize, 2.0 ** 100)
    # the sum of a softmax may be in 32 bits: an exponential (2 U) and a tree of E terms on 64 lanes (2 + 6 additions)
    assert ((w.double() - want).abs() <= (11 * U + 2.0 ** -40) * want).all(), (w, want)


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("E,k", [(4, 3), (64, 8), (200, 32)])
@pytest.mark.parametrize("lo,hi", [(-120, -88), (-709, -700), (-725, -712), (-1500, -800)])
def test_sigmoid_far_below_zero_with_a_bias(dtype, E, k, lo, hi):
    logits = (lo + (hi - lo) * torch.rand(31, E, generator=gen(E - hi), device=DEV)).to(dtype)
    check(logits, k, ffn.SCORE_SIGMOID, bias=torch.rand(E, generator=gen(E), device=DEV))


def test_sigmoid_keys_below_the_smallest_normal_number():
    """Without a difference in bias the order is that of the scores, here of e^-740 to e^-700 (5e-322 to 1e-304)."""
    logits = (-740 + 40 * torch.rand(9, 30, generator=gen(7), device=DEV))
    ids, _ = ffn.moe_route(logits, 4, ffn.SCORE_SIGMOID, bias=torch.zeros(30, device=DEV))
    assert torch.equal(ids, torch.exp(logits.double()).sort(dim=1, descending=True, stable=True).indices[:, :4].int())


@pytest.mark.parametrize("dtype", [BF, HF, F])
def test_softmax_of_experts_that_only_a_bias_chose(dtype):
    """All chosen ones are 800 to 1500 below an expert that is not among them."""
    E, k = 20, 4
    logits = (-1500 + 700 * torch.rand(40, E, generator=gen(9), device=DEV)).to(dtype)
    logits[:, 5] = 0
    bias = 10 + torch.rand(E, generator=gen(10), device=DEV)
    bias[5] = 0
    check(logits, k, ffn.SCORE_SOFTMAX, bias=bias)


@pytest.mark.parametrize("dtype", [BF, HF, F])
def test_the_lowest_value_is_a_score_of_zero(dtype):
    """The type's lowest value is what masks put in: such an expert is chosen where there are too few others, and
    its sigmoid is 0, alone or beside others."""
    low = torch.finfo(dtype).min
    logits = torch.full((4, 9), low, dtype=dtype, device=DEV)
    logits[1, 3] = -100
    logits[2, [2, 7]] = torch.tensor([-100.0, 5.0], device=DEV).to(dtype)
    logits[3, 1] = math.nan
    for bias in (None, torch.zeros(9, device=DEV)):
        ids, w = ffn.moe_route(logits, 3, ffn.SCORE_SIGMOID, bias=bias)
        assert (ids >= 0).all()
        assert (w[0] == 0).all() and w[1].tolist() == [1, 0, 0]
        assert w[2, 0] == 1 and w[2, 1:].max() < 1e-40
        assert ids[1].tolist() == [3, 0, 1] and ids[2].tolist() == [7, 2, 0]
