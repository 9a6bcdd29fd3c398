"""Blocks whose values are finite while their 32-point rotation is not: sums
that overflow to infinities of both signs turn into NaN, and a block may end up
with NaN and finite elements and no infinity at all. Its scale is 0xFF like any
block's with an element that is not finite; neighbours are untouched. Against
the oracle, bit for bit.

Pairs of the block's first eight elements, M each, add up to inf, inf, inf, -inf
and differ by 0; the next step makes inf, NaN of the first two and NaN, inf of
the others, and the one after that adds NaN to both infinities.
"""
import numpy as np
import pytest

import oracle
from datagen import bf16_bits_to_f32, f32_to_bf16_bits
from norm_util import check_operand, dev, values

pytestmark = pytest.mark.gpu

M = bf16_bits_to_f32(np.array([0x7F7F], np.uint16))[0]     # bf16's largest
PATTERN = np.array([1, 1, 1, 1, 1, 1, -1, -1], np.float32) * M


def _signs(n, rotate, seed):
    if rotate != "rand_sign_hadamard":
        return np.ones(n, np.float32)
    return np.where(oracle.rand_sign_bits(np.arange(n), seed), -1, 1).astype(np.float32)


def _source(rotate, seed1, seed0):
    """bf16 values [64, 96]: the pattern in one block along the rows and in one
    down the columns, its signs against the rotation's random ones."""
    rng = np.random.default_rng(41)
    x = values(rng, (64, 96), True)
    x[3, 32:40] = PATTERN * _signs(96, rotate, seed1)[32:40]
    x[32:40, 70] = PATTERN * _signs(64, rotate, seed0)[32:40]
    return x


def _only_nan(x):
    with np.errstate(all="ignore"):
        y = oracle.fwht32_f32(x)
    return np.isnan(y).any() and not np.isinf(y).any() and np.isfinite(y).any()


def test_the_pattern_has_nan_and_no_infinity():
    x = values(np.random.default_rng(42), (32,), True)
    x[:8] = PATTERN
    assert np.isfinite(x).all() and _only_nan(x)


@pytest.mark.parametrize("rotate", ["none", "hadamard", "rand_sign_hadamard", "hadamard16"])
@pytest.mark.parametrize("fmt,rnd", [("fp4_e2m1", "rne"), ("fp4_e2m1", "sr"), ("fp8_e4m3", "rne")])
def test_quantizers(mx, fmt, rnd, rotate):
    s1, s0 = 5, 6
    x = _source(rotate, s1, s0)
    t = dev(x, True)
    with np.errstate(all="ignore"):
        for axis, seed in ((1, s1), (0, s0)):
            q = (mx.quantize_fp8(t, axis, rotate, seed=seed) if fmt == "fp8_e4m3"
                 else mx.quantize(t, axis, rotate, rnd, seed=seed))
            check_operand(q, x, axis, rotate, rnd, seed, fmt, f"axis {axis}")
        if fmt == "fp4_e2m1":
            q1, q0 = mx.quantize_dual(t, rotate, rnd, seed1=s1, seed0=s0)
            check_operand(q1, x, 1, rotate, rnd, s1, fmt, "dual, axis 1")
            check_operand(q0, x, 0, rotate, rnd, s0, fmt, "dual, axis 0")
            for q in mx.quantize_pair(t, t, rotate, rnd, seed_a=s1, seed_b=s1):
                check_operand(q, x, 1, rotate, rnd, s1, fmt, "pair")


@pytest.mark.parametrize("rotate", ["none", "hadamard", "rand_sign_hadamard", "hadamard16"])
@pytest.mark.parametrize("fmt,rnd", [("fp4_e2m1", "rne"), ("fp4_e2m1", "sr"), ("fp8_e4m3", "rne")])
def test_norm(mx, fmt, rnd, rotate):
    """The same through the norm, whose weight lifts eight columns to M (and one
    more for the block down the columns)."""
    s1, s0 = 5, 6
    rng = np.random.default_rng(43)
    x = np.where(rng.random((64, 96)) < 0.5, -1, 1).astype(np.float32)
    x[3, 32:40] = np.sign(PATTERN) * _signs(96, rotate, s1)[32:40]
    x[32:40, 70] = np.sign(PATTERN) * _signs(64, rotate, s0)[32:40]
    x[:32, 70] = x[40:, 70] = 0.0
    w = np.ones(96, np.float32)
    w[32:40] = w[70] = np.float32(3.3e38)
    with np.errstate(all="ignore"):
        h, rstd, y = oracle.rmsnorm_ref(x, w, None, 0.0, True)
        assert np.isfinite(y).all()
        for dual in (False, True):
            got = mx.rmsnorm_quantize(dev(x, True), dev(w, False), eps=0.0, format=fmt, dual=dual,
                                      rotate=rotate, round=rnd, seed1=s1, seed0=s0)
            check_operand(got.q1, y, 1, rotate, rnd, s1, fmt, f"axis 1, dual {dual}")
            if dual:
                check_operand(got.q0, y, 0, rotate, rnd, s0, fmt, "axis 0")
