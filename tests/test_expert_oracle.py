"""Pins of the oracle of the epilogues and the grouped quantizer. No GPU."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

import oracle
from datagen import normal_bf16

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
TORCH = {"none": lambda z: z, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
         "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}


@pytest.mark.parametrize("act", ACTS)
def test_activation_and_slope(act):
    z = np.concatenate([np.linspace(-30, 30, 1201), np.random.default_rng(1).normal(size=500)])
    t = torch.tensor(z, requires_grad=True)
    y = TORCH[act](t)
    y.sum().backward()
    got, slope = oracle.act_ref(z, act)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-14)
    keep = z != 0                                   # relu's slope at 0 is a choice: 0
    assert np.allclose(slope[keep], t.grad.numpy()[keep], rtol=1e-12, atol=1e-13)
    assert act != "relu" or slope[~keep] == 0


@pytest.mark.parametrize("act", ACTS)
def test_epilogue_and_its_gradient(act):
    rng = np.random.default_rng(2)
    acc, mul, res, up = (torch.tensor(rng.normal(size=(7, 5))) for _ in range(4))
    bias = torch.tensor(rng.normal(size=5))
    pre = (acc + bias).requires_grad_()
    m = mul.clone().requires_grad_()
    c = TORCH[act](pre) * m + res
    c.backward(up)
    got, z = oracle.epilogue_ref(acc.numpy(), act, bias.numpy(), mul.numpy(), res.numpy())
    assert np.allclose(got, c.detach().numpy(), rtol=1e-12)
    assert np.allclose(z, pre.detach().numpy(), rtol=1e-15)
    dz, dmul = oracle.act_backward_ref(up.numpy(), z, act, mul.numpy())
    assert np.allclose(dz, pre.grad.numpy(), rtol=1e-11, atol=1e-14)
    assert np.allclose(dmul, m.grad.numpy(), rtol=1e-11, atol=1e-14)


def test_group_ranges():
    assert oracle.group_ranges_ref([2, 2, 5], 5) == [(0, 2), (2, 2), (2, 5)]
    assert oracle.group_ranges_ref([3, 1, 9, -4], 6) == [(0, 3), (3, 3), (3, 6), (6, 6)]
    assert oracle.group_ranges_ref([-1, 0], 4) == [(0, 0), (0, 0)]
    assert oracle.grouped_slices_ref(1000, 3) == 10
    assert oracle.grouped_slices_ref(600, 3, 200) == 6


@pytest.mark.parametrize("rotate", ["none", "hadamard", "rand_sign_hadamard", "hadamard16"])
def test_grouped_quantize_is_each_group_padded(rotate):
    rng = np.random.Generator(np.random.PCG64(3))
    x = normal_bf16(rng, (300, 64))
    ranges = [(0, 40), (40, 40), (40, 233)]
    (c1, s1), (c0, s0) = oracle.grouped_quantize_ref(x, ranges, 5, rotate, "rne", 7, 7)
    q = oracle.quantize_ref(x, 1, rotate=rotate, seed=7)
    got = oracle.untile_codes(c1, 300, 64)
    assert np.array_equal(got[:233], q.codes[:233]) and not got[233:].any()
    assert np.array_equal(oracle.untile_scales(s1, 300, 64)[:233], q.scales[:233])
    codes, scales = oracle.untile_codes(c0, 64, 640), oracle.untile_scales(s0, 64, 640)
    for (first, last), at in zip(ranges, (0, 128, 128)):
        n = last - first
        deep = -(-n // 32) * 32
        part = np.zeros((deep, 64), np.uint16)
        part[:n] = x[first:last]
        if n:
            q = oracle.quantize_ref(part, 0, rotate=rotate, seed=7)
            assert np.array_equal(codes[:, at:at + deep], q.codes)
            assert np.array_equal(scales[:, at // 32:(at + deep) // 32], q.scales)
    assert not codes[:, 128 + 224:].any()
