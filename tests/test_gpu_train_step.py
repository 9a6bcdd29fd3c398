"""The norm, the linears, the norm's gradient and clipping together, as a
training step of two quantized linears with a residual path runs them:

    h = x + res;  y = norm(h);  a = y W1^T;  z = a W2^T;  out = h + z

forward, backward from d(out), then clipping of the three weight gradients.
Every call is checked against the oracle fed with that call's own inputs (the
GPU's outputs of the step before), so each bound is that call's: operands bit
for bit, products within the linears' 1e-5, gradients within fp32 rounding.
"""
import numpy as np
import pytest

import oracle
from norm_util import check_operand, dev, host, values

pytestmark = pytest.mark.gpu

T, D, F = 256, 192, 320
SEEDS = {"seed_a": 21, "seed_b": 21 | 1 << 32}


def _gemm(qa, qb, c, axes, fmt):
    """Relative error of the product of two packed operands against fp64."""
    def values_of(q):
        mn, k = q.mn, q.k
        codes = (oracle.untile_codes_fp8 if fmt == "fp8_e4m3" else oracle.untile_codes)(
            q.codes.cpu().numpy(), mn, k)
        return oracle.dequantize_ref(codes, oracle.untile_scales(q.scales.cpu().numpy(), mn, k), fmt)
    assert (qa.axis, qb.axis) == axes
    ref = values_of(qa) @ values_of(qb).T
    return np.linalg.norm(host(c) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("fmt,rotate,rnd", [("fp4_e2m1", "hadamard", "rne"),
                                            ("fp4_e2m1", "rand_sign_hadamard", "sr"),
                                            ("fp8_e4m3", "hadamard16", "rne")])
def test_training_step(mx, fmt, rotate, rnd):
    import torch
    rng = np.random.default_rng(31)
    tol = 1e-5 if fmt == "fp4_e2m1" else 1e-4   # see the linears' own tests
    sa, sb = SEEDS["seed_a"], SEEDS["seed_b"]
    x, res = dev(values(rng, (T, D), True), True), dev(values(rng, (T, D), True), True)
    g = dev(np.abs(values(rng, (D,), False)) + 0.5, False)
    w1, w2 = dev(values(rng, (F, D), True, .05), True), dev(values(rng, (D, F), True, .05), True)
    dout = dev(values(rng, (T, D), True, 1e-3), True)

    def quant(t, axis, seed):
        if fmt == "fp8_e4m3":
            return mx.quantize_fp8(t, axis, rotate, seed=seed)
        return mx.quantize(t, axis, rotate, rnd, seed=seed)

    # forward
    n = mx.rmsnorm_quantize(x, g, res, format=fmt, dual=True, rotate=rotate, round=rnd, seed1=sa,
                            seed0=sb)
    h, rstd, y = oracle.rmsnorm_ref(host(x), host(g), host(res), 1e-5, True)
    assert np.array_equal(host(n.h), h) and np.array_equal(host(n.rstd), rstd)
    check_operand(n.q1, y, 1, rotate, rnd, sa, fmt, "y axis 1")
    check_operand(n.q0, y, 0, rotate, rnd, sb, fmt, "y axis 0")
    qw1 = quant(w1, 1, sb)
    a = mx.linear("fprop", n.q1, qw1, "bf16")
    assert _gemm(n.q1, qw1, mx.linear("fprop", n.q1, qw1), (1, 1), fmt) <= tol
    qa, qw2 = quant(a, 1, sa), quant(w2, 1, sb)
    z = mx.linear("fprop", qa, qw2, "bf16")
    out = n.h + z

    # backward: out = h + z, so dout reaches h past the linears too
    da = mx.linear("dgrad", quant(dout, 1, sa), quant(w2, 0, sb), "bf16")
    dw2 = mx.linear("wgrad", quant(dout, 0, sa), quant(a, 0, sb))
    qda1, qda0 = quant(da, 1, sa), quant(da, 0, sa)
    dy = mx.linear("dgrad", qda1, quant(w1, 0, sb), "bf16")
    dw1 = mx.linear("wgrad", qda0, n.q0)
    assert _gemm(qda0, n.q0, dw1, (0, 0), fmt) <= tol
    dh, dg = mx.rmsnorm_backward(dy, n.h, n.rstd, g, dres=dout)
    rh, rg = oracle.rmsnorm_backward_ref(host(dy), h, rstd, host(g), host(dout))
    # bf16's half step 2^-8 of the result and fp32's error of the terms: their
    # largest magnitudes stand in for each element's own
    scale = np.abs(host(dy) * host(g)).max() * np.abs(rstd).max() * (1 + np.abs(h * rstd[:, None]).max() ** 2)
    assert np.all(np.abs(host(dh) - rh) <= 2.0 ** -8 * 1.001 * np.abs(rh) + 128 * 2.0 ** -24 * scale)
    terms = np.abs(host(dy) * h * rstd[:, None]).sum(0)
    assert np.all(np.abs(host(dg) - rg) <= 72 * 2.0 ** -24 * terms + 1e-30)

    # clipping: fp32 matrices as the linears wrote them, the vector from the norm
    grads = [dw1, dw2, dg]
    before = [host(t).copy() for t in grads]
    norm, ref = oracle.clip_ref(before, 0.01)
    assert norm > 0.01
    got = mx.clip_grad_norm(mx.GradSet(grads), 0.01)
    assert abs(float(got) - norm) <= 1.001 * 2.0 ** -24 * norm
    for t, r in zip(grads, ref):
        assert np.all(np.abs(host(t) - r) <= 2.002 * 2.0 ** -24 * np.abs(r) + 2.0 ** -149)
    assert torch.isfinite(out).all()


def test_step_captured_twice(mx):
    """Forward, gradient and clipping captured as two graphs over the same
    weights, replayed in turn with eager steps between: the eager step's bytes
    every time."""
    import torch
    rng = np.random.default_rng(32)
    g = dev(np.abs(values(rng, (D,), False)) + 0.5, False)
    qw = mx.quantize(dev(values(rng, (F, D), True, .05), True), 1, seed=1 << 32)
    qw0 = mx.quantize(dev(values(rng, (F, D), True, .05), True), 0, seed=1 << 32)
    ins = [(dev(values(rng, (T, D), True), True), dev(values(rng, (T, D), True), True),
            dev(values(rng, (T, F), True, 1e-3), True)) for _ in range(2)]
    bufs = [[torch.zeros(F, D, device="cuda"), torch.zeros(D, device="cuda")] for _ in range(3)]
    sets = [mx.GradSet(b) for b in bufs]

    def step(x, r, dout, i):
        n = mx.rmsnorm_quantize(x, g, r, dual=True, seed0=1 << 32)
        out = mx.linear("fprop", n.q1, qw, "bf16")
        dy = mx.linear("dgrad", mx.quantize(dout, 1), qw0, "bf16")
        mx.linear("wgrad", mx.quantize(dout, 0), n.q0, out=bufs[i][0])
        dh, dg = mx.rmsnorm_backward(dy, n.h, n.rstd, g)
        bufs[i][1].copy_(dg)
        norm = mx.clip_grad_norm(sets[i], 0.01)
        return [out, n.h, dh, norm, *bufs[i]]

    step(*ins[0], 2)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(*ins[i], i))
        graphs.append(graph)
    for k in range(3):
        for x, r, dout in ins:
            x.copy_(dev(values(rng, (T, D), True), True))
            dout.copy_(dev(values(rng, (T, F), True, 1e-3), True))
        for i in (0, 1):
            graphs[i].replay()
        for i in (1, 0):
            want = step(*ins[i], 2)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want)), (k, i)
