"""Plain CPU oracle of the epilogues, the grouped products and the grouped
quantizer (NumPy, fp64) -- TEST INFRASTRUCTURE ONLY, like the rest of this
package.

What pins each function (tests/test_expert_oracle.py, "not gpu"):
  act_ref              torch's float64 activations and their autograd.
  epilogue_ref,
  act_backward_ref     torch autograd in float64.
  group_ranges_ref     worked examples.
  grouped_quantize_ref quantize_ref of every group by itself, padded.
"""
from __future__ import annotations

from typing import List, Tuple

import numpy as np

from .mx_oracle import quantize_ref, rand_sign_bits, tile_codes, tile_scales

__all__ = ["act_ref", "epilogue_ref", "act_backward_ref", "group_ranges_ref", "grouped_slices_ref",
           "grouped_quantize_ref"]


def _erf(x: np.ndarray) -> np.ndarray:
    from scipy.special import erf
    return erf(x)


def act_ref(z: np.ndarray, act: str) -> Tuple[np.ndarray, np.ndarray]:
    """(act(z), act'(z)) in fp64."""
    z = np.asarray(z, np.float64)
    with np.errstate(over="ignore"):
        if act == "none":
            return z, np.ones_like(z)
        if act == "relu":
            return np.maximum(z, 0.0), np.where(np.isnan(z), z, np.where(z > 0, 1.0, 0.0))
        if act == "gelu":
            cdf = 0.5 * (1.0 + _erf(z / np.sqrt(2.0)))
            return z * cdf, cdf + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
        if act == "silu":
            u, du = z, 1.0
        elif act == "gelu_tanh":
            c = np.sqrt(2.0 / np.pi)
            u, du = 2.0 * c * (z + 0.044715 * z ** 3), 2.0 * c * (1.0 + 3 * 0.044715 * z * z)
        else:
            raise ValueError(act)
        p = 1.0 / (1.0 + np.exp(-u))
        return z * p, p + z * p * (1.0 - p) * du


def epilogue_ref(acc, act: str = "none", bias=None, mul=None, residual=None):
    """(C, pre) in fp64."""
    pre = np.asarray(acc, np.float64) + (0.0 if bias is None else np.asarray(bias, np.float64))
    c = act_ref(pre, act)[0]
    if mul is not None:
        c = c * np.asarray(mul, np.float64)
    if residual is not None:
        c = c + np.asarray(residual, np.float64)
    return c, pre


def act_backward_ref(acc, pre, act: str, mul=None):
    """(gradient of pre, gradient of mul) in fp64."""
    y, slope = act_ref(pre, act)
    m = 1.0 if mul is None else np.asarray(mul, np.float64)
    return acc * m * slope, acc * y


def group_ranges_ref(ends, rows: int) -> List[Tuple[int, int]]:
    """[first, last) of each group: an end below an earlier one counts as that
    one, one past the last row as the last row."""
    out, at = [], 0
    for e in ends:
        last = max(at, min(max(int(e), 0), rows))
        out.append((at, last))
        at = last
    return out


def grouped_slices_ref(rows: int, groups: int, group_rows: int = -1) -> int:
    return (rows + 127 * groups) // 128 if group_rows < 0 else groups * -(-group_rows // 128)


def grouped_quantize_ref(x_bits: np.ndarray, ranges, slices: int, rotate: str, rounding: str,
                         seed1: int, seed0: int):
    """((codes, scales) of axis 1, (codes, scales) of the grouped axis-0 operand),
    packed, of bf16 rows in the order of the groups."""
    rows, cols = x_bits.shape
    live = ranges[-1][1]
    q1 = quantize_ref(x_bits[:live], 1, rotate=rotate, rounding=rounding, seed=seed1)
    c1, s1 = np.zeros((rows, cols), np.uint8), np.zeros((rows, cols // 32), np.uint8)
    c1[:live], s1[:live] = q1.codes, q1.scales
    c0, s0 = np.zeros((cols, 128 * slices), np.uint8), np.zeros((cols, 4 * slices), np.uint8)
    at = 0
    for first, last in ranges:
        n = last - first
        deep = -(-n // 32) * 32
        if n:
            part = np.zeros((deep, cols), np.uint16)
            part[:n] = x_bits[first:last]
            rot = rotate
            if rotate == "rand_sign_hadamard":       # signs by the place within the group
                sign = rand_sign_bits(np.arange(deep), seed0).astype(np.uint16) << np.uint16(15)
                part ^= sign[:, None]
                rot = "hadamard"
            q = quantize_ref(part, 0, rotate=rot, rounding=rounding, seed=seed0,
                             row_index=first + np.arange(deep))
            c0[:, at:at + deep], s0[:, at // 32:(at + deep) // 32] = q.codes, q.scales
        at += -(-n // 128) * 128
    return (tile_codes(c1), tile_scales(s1, cols)), (tile_codes(c0), tile_scales(s0, 128 * slices))
