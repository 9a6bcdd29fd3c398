"""Pins of the norm, gradient and clipping oracle against torch in float64,
central differences and exact fractions. CPU only."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from datagen import bf16_bits_to_f32, f32_to_bf16_bits


def test_rmsnorm_matches_float64():
    rng = np.random.default_rng(0)
    x, r = rng.standard_normal((2, 5, 96)).astype(np.float32)
    w = rng.standard_normal(96).astype(np.float32)
    h, rstd, y = oracle.rmsnorm_ref(x, w, r, 1e-5, bf16=False)
    t = torch.from_numpy(x.astype(np.float64)) + torch.from_numpy(r.astype(np.float64))
    assert np.abs(h - t.numpy()).max() <= 2.0 ** -24 * np.abs(t.numpy()).max()
    t = torch.from_numpy(h.astype(np.float64))
    ref = t / torch.sqrt(t.square().mean(1, keepdim=True) + 1e-5) * torch.from_numpy(w).double()
    # rstd, the product with it and the one with the weight each round once
    assert np.all(np.abs(y - ref.numpy()) <= 3.01 * 2.0 ** -24 * np.abs(ref.numpy()))
    assert rstd.dtype == np.float32


def test_rmsnorm_stream_is_bf16_and_worked_rows():
    x = np.array([[1.0, 3.0] * 16, [0.0] * 32], np.float32)
    r = np.array([[2.0 ** -9, 2.0 ** -8] * 16, [0.0] * 32], np.float32)
    h, rstd, y = oracle.rmsnorm_ref(x, np.ones(32), r, 0.0, bf16=True)
    # 1 + 2^-9 lies below half of bf16's step 2^-7 at 1; 3 + 2^-8 below half of 2^-6
    assert np.array_equal(h[0], x[0])
    assert rstd[0] == np.float32(1 / np.sqrt(5.0))
    assert np.isinf(rstd[1]) and np.isnan(y[1]).all()       # 0 / 0 without an eps
    h, rstd, y = oracle.rmsnorm_ref(x, np.ones(32), r, 0.25, bf16=True)
    assert rstd[1] == 2.0 and not y[1].any()


def test_fp32_sum_of_bf16_rounds_like_the_exact_sum():
    """The stream's bf16 sum is formed in fp32 first: over every distance of
    exponents the two roundings equal the exact sum's one rounding."""
    rng = np.random.default_rng(1)
    m = rng.integers(128, 256, 4000)
    n = rng.integers(128, 256, 4000) * rng.choice([-1, 1], 4000)
    for d in range(0, 40):
        a, b = m.astype(np.float64) * 2.0 ** d, n.astype(np.float64)
        one = bf16_bits_to_f32(f32_to_bf16_bits(a.astype(np.float32) + b.astype(np.float32)))
        exact = a + b                                        # 48 bits at most
        q = np.exp2(np.floor(np.log2(np.maximum(np.abs(exact), 1e-9))) - 7)
        assert np.array_equal(one, np.round(exact / q) * q), d


def test_backward_matches_autograd_and_differences():
    rng = np.random.default_rng(2)
    h, dy, dres, d = rng.standard_normal((4, 6, 64))
    w = rng.standard_normal(64)
    eps = 1e-3
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    th = torch.tensor(h, requires_grad=True)
    tw = torch.tensor(w, requires_grad=True)
    y = th / torch.sqrt(th.square().mean(1, keepdim=True) + eps) * tw
    ((y * torch.tensor(dy)).sum() + (th * torch.tensor(dres)).sum()).backward()
    dh, dw = oracle.rmsnorm_backward_ref(dy, h, rstd, w, dres)
    assert np.allclose(dh, th.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dw, tw.grad.numpy(), rtol=1e-12, atol=1e-12)

    def loss(hh, ww):
        return ((hh / np.sqrt((hh * hh).mean(1, keepdims=True) + eps) * ww) * dy).sum() \
            + (hh * dres).sum()

    t = 1e-5
    assert abs((loss(h + t * d, w) - loss(h - t * d, w)) / (2 * t) - (dh * d).sum()) < 1e-7
    e = rng.standard_normal(64)
    assert abs((loss(h, w + t * e) - loss(h, w - t * e)) / (2 * t) - (dw * e).sum()) < 1e-7


@pytest.mark.parametrize("max_norm", [0.5, 7.0, 1e6, 0.0])
def test_clip_matches_torch(max_norm):
    rng = np.random.default_rng(3)
    grads = [rng.standard_normal(s) for s in ((3, 5), (7,), (1, 1))]
    params = [torch.nn.Parameter(torch.zeros(g.shape, dtype=torch.float64)) for g in grads]
    for p, g in zip(params, grads):
        p.grad = torch.tensor(g)
    want = torch.nn.utils.clip_grad_norm_(params, max_norm)
    norm, out = oracle.clip_ref(grads, max_norm)
    assert abs(norm - float(want)) < 1e-12
    for o, p in zip(out, params):
        assert np.allclose(o, p.grad.numpy(), rtol=1e-12, atol=0)


def test_grad_norm_exact_and_nonfinite():
    grads = [np.array([3, 4, 12]), np.array([[84]])]
    assert Fraction(oracle.grad_norm_ref(grads)) == Fraction(85)
    norm, out = oracle.clip_ref([np.array([1.0, np.inf])], 1.0)
    assert norm == np.inf and out[0][0] == 0 and np.isnan(out[0][1])
    norm, out = oracle.clip_ref([np.array([1.0, np.nan])], 1.0)
    assert np.isnan(norm) and np.isnan(out[0]).all()
