"""Helpers of the tests of epilogues and grouped products: operands with their
fp64 values, and how far an output may be off.

A sum acc of K products is within (K / 128 + 10) 2^-22 S of the exact one, S
the sum of the products' magnitudes: one instruction adds 128 exact products to
an fp32 sum, keeping some bits more than fp32's 24 of the largest of them (2^-22
of S covers a truncation of each operand as well), and at most eight partial
sums are added. From there U = 2^-24 for each fp32 operation; an activation is
within 2^-20 (1 + |z|) (the logistic's argument is off by at most 3 U |z|,
which moves z p by at most 3 U z^2 p (1 - p) < 2 U; exp2 and the reciprocal
are off by 2 U each; the GELU's erfc is off by 1.5e-7, half of it times |z|
counts), a slope within 2^-19; activations move by at most 1.13 times what z
does.
"""
import numpy as np

import oracle

U = 2.0 ** -24
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def values(q, axis=None):
    """fp64 values [MN, K] of an operand, K padded for a grouped one."""
    mn = q.mn
    k = q.k
    if q.axis == 2:
        k = 128 * oracle.grouped_slices_ref(q.desc.rows, q.groups, q.group_rows)
    if mn == 0 or k == 0 or q.codes.numel() == 0:
        return np.zeros((mn, k))
    codes = oracle.untile_codes(q.codes.cpu().numpy(), mn, k)
    return oracle.dequantize_ref(codes, oracle.untile_scales(q.scales.cpu().numpy(), mn, k))


def product(a, b):
    """(acc, its bound) of K-major values."""
    return a @ b.T, (a.shape[1] / 128 + 10) * 2.0 ** -22 * (np.abs(a) @ np.abs(b).T)


def host64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(got, ref, bound, dtype, what):
    got = host64(got)
    bound = bound + STEP[dtype] * (np.abs(ref) + bound) + 2.0 ** -133
    off = np.abs(got - ref)
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(off / bound)} of its bound at {np.argwhere(bad)[0]}")


def check_forward(got, pre, acc, err, dtype, act, bias, mul, residual, what):
    c, z = oracle.epilogue_ref(acc, act, bias, mul, residual)
    err = err + U * np.abs(z)
    if pre is not None:
        check(pre, z, err, dtype, what + " pre")
    y = oracle.act_ref(z, act)[0]
    if act != "none":
        err = 1.13 * err + 2.0 ** -20 * (1 + np.abs(z))
    if mul is not None:
        err = np.abs(mul) * err + U * np.abs(y * mul)
    if residual is not None:
        err = err + U * np.abs(c)
    check(got, c, err, dtype, what)


def check_backward(dz, dmul, acc, err, pre, dtype, act, mul, what):
    y, slope = oracle.act_ref(pre, act)
    ref, refmul = oracle.act_backward_ref(acc, pre, act, mul)
    m = 1.0 if mul is None else np.abs(mul)
    check(dz, ref, (err * np.abs(slope) + np.abs(acc) * 2.0 ** -19) * m + 2 * U * np.abs(ref),
          dtype, what + " dz")
    if mul is not None:
        check(dmul, refmul, err * np.abs(y) + np.abs(acc) * 2.0 ** -20 * (1 + np.abs(pre))
              + U * np.abs(refmul), dtype, what + " dmul")
