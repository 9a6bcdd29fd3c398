"""Plain CPU oracle of the norm, its gradient and clipping by the global norm
(NumPy, sums in fp64) -- TEST INFRASTRUCTURE ONLY, like the rest of this
package.

rmsnorm_ref takes each rounding where the operator defines one: the stream h
to its own type, rstd once from fp64, and y by two fp32 products; its y then
goes through quantize_values_ref. The others are fp64 throughout: the tests
derive how far fp32 kernels may be from them.

What pins each function (tests/test_norm_oracle.py, "not gpu"):
  rmsnorm_ref           torch's float64 norm of the same rows; worked rows.
  rmsnorm_backward_ref  torch autograd in float64, and central differences of
                        rmsnorm_ref's formula.
  grad_norm_ref,
  clip_ref              torch.nn.utils.clip_grad_norm_ in float64; exact
                        fractions on small integers.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import numpy as np

from .mx_oracle import bf16_round_ref

__all__ = ["rmsnorm_ref", "rmsnorm_backward_ref", "grad_norm_ref", "clip_ref"]

CLIP_EPS = 1e-6


def rmsnorm_ref(x: np.ndarray, weight: np.ndarray, residual: Optional[np.ndarray], eps: float,
                bf16: bool) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(h, rstd, y) of fp32 arrays; bf16: the stream is stored in bf16 (x and
    residual then hold bf16 values)."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        h = x if residual is None else x + np.asarray(residual, np.float32)
        if residual is not None and bf16:
            h = (bf16_round_ref(h).astype(np.uint32) << 16).view(np.float32)
        h64 = h.astype(np.float64)
        rstd = (1.0 / np.sqrt((h64 * h64).mean(axis=1) + eps)).astype(np.float32)
        y = (h * rstd[:, None]).astype(np.float32) * np.asarray(weight, np.float32)[None, :]
    return h, rstd, y.astype(np.float32)


def rmsnorm_backward_ref(dy, h, rstd, weight, dres=None) -> Tuple[np.ndarray, np.ndarray]:
    """(dh, dweight) in fp64."""
    dy, h, w = (np.asarray(v, np.float64) for v in (dy, h, weight))
    xhat = h * np.asarray(rstd, np.float64)[:, None]
    g = dy * w[None, :]
    dh = (g - xhat * (g * xhat).mean(axis=1, keepdims=True)) * np.asarray(rstd, np.float64)[:, None]
    if dres is not None:
        dh = dh + np.asarray(dres, np.float64)
    return dh, (dy * xhat).sum(axis=0)


def grad_norm_ref(grads: Sequence[np.ndarray]) -> float:
    return float(np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads)))


def clip_ref(grads: Sequence[np.ndarray], max_norm: float):
    """(norm, clipped tensors in fp64)."""
    norm = grad_norm_ref(grads)
    with np.errstate(all="ignore"):
        coef = np.minimum(1.0, np.float64(max_norm) / (norm + CLIP_EPS))   # NaN stays NaN
        if np.isinf(max_norm) and not np.isnan(norm):
            coef = 1.0                                                     # no limit
        return norm, [np.asarray(g, np.float64) * coef for g in grads]
