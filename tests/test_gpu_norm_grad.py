"""Gradient of the RMS norm on the GPU against the oracle in fp64.

The bounds, with u = 2^-24 and half a step s of the output's type (2^-8 for
bf16, u for fp32), n columns: x^ = h * rstd and dy * weight round once each;
their products are added up in fp32 in chains of at most
K = n / 512 + 64 additions (a thread's columns, the wave, the waves), so the
mean is off by (K + 4) u of the mean of the magnitudes S; the result's own
products and sums round three more times. Hence per element

    |dh - ref| <= rstd (6 u (|dy w| + |x^ m|) + |x^| (K + 4) u S)
                  + 2 u (|dres| + |ref|) + s |ref| + half the smallest subnormal

and a weight gradient, added over R rows in chains of at most R / 64 + 64
(fp32 within a workgroup, fp64 across them), is within
(R / 64 + 68) u sum |dy x^|. Both have u times 1.01 for the products of
roundings.
"""
import numpy as np
import pytest

import oracle
from norm_util import dev, host, values

pytestmark = pytest.mark.gpu

U = 1.01 * 2.0 ** -24


def _inputs(rows, cols, bf16, wbf16, dres, seed=0):
    rng = np.random.default_rng(rows * 17 + cols + seed)
    h = values(rng, (rows, cols), bf16)
    dy = values(rng, (rows, cols), bf16, 1e-4)
    w = values(rng, (cols,), wbf16)
    d = values(rng, (rows, cols), bf16, 1e-4) if dres else None
    rstd = (1 / np.sqrt((h.astype(np.float64) ** 2).mean(1) + 1e-5)).astype(np.float32)
    return dy, h, rstd, w, d


def _check(got, dy, h, rstd, w, d, bf16):
    rows, cols = dy.shape
    dh, dw = oracle.rmsnorm_backward_ref(dy, h, rstd, w, d)
    rs = np.abs(rstd.astype(np.float64))[:, None]
    xh = np.abs(h.astype(np.float64)) * rs
    g = np.abs(dy.astype(np.float64) * w)
    S = (g * xh).mean(1, keepdims=True)
    m = np.abs((dy.astype(np.float64) * w * h * rstd[:, None]).mean(1, keepdims=True))
    K = cols / 512 + 64
    step, tiny = (2.0 ** -8, 2.0 ** -134) if bf16 else (2.0 ** -24, 2.0 ** -150)
    bound = rs * (6 * U * (g + xh * m) + xh * (K + 4) * U * S) + (2 * U + step) * np.abs(dh) + tiny
    if d is not None:
        bound += 2 * U * np.abs(d)
    err = np.abs(host(got[0]).astype(np.float64) - dh)
    assert np.all(err <= bound), f"dh: {(err / bound).max():.3g} of the bound"
    limit = (rows / 64 + 68) * U * (np.abs(dy.astype(np.float64)) * xh).sum(0) + 2.0 ** -150
    err = np.abs(host(got[1]).astype(np.float64) - dw)
    assert np.all(err <= limit), f"dweight: {(err / limit).max():.3g} of the bound"


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (3, 40), (32, 512), (64, 1024),
                                       (8, 4096), (9, 4096), (31, 1000), (32, 1024), (33, 512), (16, 2048),
                                       (1, 4104), (2, 16), (777, 1056),
                                       (1100, 328), (2048, 4096), (65, 8192), (40, 14336),
                                       (9, 16416), (700, 40008), (5000, 64), (6000, 4096)])
@pytest.mark.parametrize("bf16", [True, False])
def test_against_oracle(mx, rows, cols, bf16):
    for dres, wbf16 in ((True, bf16), (False, not bf16)):
        dy, h, rstd, w, d = _inputs(rows, cols, bf16, wbf16, dres)
        got = mx.rmsnorm_backward(dev(dy, bf16), dev(h, bf16), dev(rstd, False), dev(w, wbf16),
                                  None if d is None else dev(d, bf16))
        _check(got, dy, h, rstd, w, d, bf16)


def test_against_differences(mx):
    """Directional derivatives of the norm's formula in fp64. fp32 gradients of
    2048 terms each are within the bound above of the formula's; the central
    difference adds t^2 / 6 of the third derivative, below 1e-9 of the sum."""
    rng = np.random.default_rng(5)
    rows, cols, eps = 8, 256, 1e-5
    dy, h, _, w, d = _inputs(rows, cols, False, False, True)
    rstd = (1 / np.sqrt((h.astype(np.float64) ** 2).mean(1) + eps)).astype(np.float32)
    dh, dw = mx.rmsnorm_backward(dev(dy, False), dev(h, False), dev(rstd, False), dev(w, False),
                                 dev(d, False))

    def loss(hh, ww):
        r = 1 / np.sqrt((hh * hh).mean(1, keepdims=True) + eps)
        return (hh * r * ww * dy).sum() + (hh * d).sum()

    h, w, dy, d = (v.astype(np.float64) for v in (h, w, dy, d))
    t = 1e-4
    e = rng.standard_normal(h.shape)
    diff = (loss(h + t * e, w) - loss(h - t * e, w)) / (2 * t)
    terms = np.abs(host(dh) * e).sum()
    assert abs(diff - (host(dh).astype(np.float64) * e).sum()) <= 1e-5 * terms
    e = rng.standard_normal(w.shape)
    diff = (loss(h, w + t * e) - loss(h, w - t * e)) / (2 * t)
    assert abs(diff - (host(dw).astype(np.float64) * e).sum()) <= 1e-5 * np.abs(host(dw) * e).sum()


@pytest.mark.parametrize("cols", [64, 4096, 40008])
def test_strided_and_in_place(mx, cols):
    import torch
    for bf16 in (True, False):
        dy, h, rstd, w, d = _inputs(21, cols, bf16, True, True)
        ld = cols + 16
        want = mx.rmsnorm_backward(dev(dy, bf16), dev(h, bf16), dev(rstd, False), dev(w, True),
                                   dev(d, bf16))
        big = torch.full((30, ld), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32,
                         device="cuda")
        got = mx.rmsnorm_backward(dev(dy, bf16, ld), dev(h, bf16, ld), dev(rstd, False),
                                  dev(w, True), dev(d, bf16, ld), dh=big[4:25, 8:8 + cols])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        big[4:25, 8:8 + cols] = 7.0
        assert torch.all(big == 7.0)
        for over in (0, 1):
            a, b = dev(dy, bf16), dev(d, bf16)
            got = mx.rmsnorm_backward(a, dev(h, bf16), dev(rstd, False), dev(w, True), b,
                                      dh=(a, b)[over])
            assert got[0] is (a, b)[over]
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_beyond_32_bits(mx):
    import torch
    rows, cols, ld = 64, 256, 1 << 26
    big = torch.empty((rows * ld,), dtype=torch.bfloat16, device="cuda").view(rows, ld)
    parts = [big[:, k * 1024:k * 1024 + cols] for k in range(4)]
    dy, h, rstd, w, d = _inputs(rows, cols, True, True, True)
    for p, v in zip(parts, (dy, h, d)):
        p.copy_(dev(v, True))
    got = mx.rmsnorm_backward(parts[0], parts[1], dev(rstd, False), dev(w, True), parts[2],
                              dh=parts[3])
    _check(got, dy, h, rstd, w, d, True)


@pytest.mark.parametrize("rows,cols", [(1, 4096), (8, 4096), (16, 2048), (32, 1024), (32, 512)])
def test_few_rows_in_place(mx, rows, cols):
    """Few rows take one launch, whose workgroups all read the whole of dy: over
    dy, over dres and beside both give the same dh, and so does dweight."""
    import torch
    for bf16 in (True, False):
        dy, h, rstd, w, d = _inputs(rows, cols, bf16, True, True)
        rest = dev(h, bf16), dev(rstd, False), dev(w, True)
        want = mx.rmsnorm_backward(dev(dy, bf16), *rest, dev(d, bf16))
        for _ in range(20):
            a, b = dev(dy, bf16), dev(d, bf16)
            got = mx.rmsnorm_backward(a, *rest, b, dh=a)
            assert got[0] is a and torch.equal(a, want[0]) and torch.equal(got[1], want[1])
            a = dev(dy, bf16)
            got = mx.rmsnorm_backward(a, *rest, b, dh=b)
            assert got[0] is b and torch.equal(b, want[0]) and torch.equal(got[1], want[1])


def test_deterministic_and_nonfinite(mx):
    import torch
    dy, h, rstd, w, d = _inputs(1500, 520, True, True, True)
    args = dev(dy, True), dev(h, True), dev(rstd, False), dev(w, True), dev(d, True)
    a, b = mx.rmsnorm_backward(*args), mx.rmsnorm_backward(*args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dy[7, 3] = np.nan                          # its row, and its column of dweight
    dh, dw = mx.rmsnorm_backward(dev(dy, True), *args[1:])
    assert torch.isnan(dh[7]).all() and torch.isnan(dw[3])
    keep = torch.arange(1500, device="cuda") != 7
    assert torch.equal(dh[keep], a[0][keep])
    assert torch.isfinite(dw[torch.arange(520, device="cuda") != 3]).all()


def test_empty(mx):
    import torch
    z = torch.empty((0, 64), device="cuda")
    dh, dw = mx.rmsnorm_backward(z, z, torch.empty(0, device="cuda"), torch.ones(64, device="cuda"))
    assert dh.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device="cuda"))
    z = torch.empty((5, 0), device="cuda")
    dh, dw = mx.rmsnorm_backward(z, z, torch.ones(5, device="cuda"), torch.empty(0, device="cuda"))
    assert dw.numel() == 0


def test_streams_and_graphs(mx):
    """On a side stream, and two captured calls replayed in turn with eager
    calls between: each has its own workspace."""
    import torch
    cases = [_inputs(300, 512, True, True, True, s) for s in (1, 2)]
    dev_args = [[dev(c[0], True), dev(c[1], True), dev(c[2], False), dev(c[3], True),
                 dev(c[4], True)] for c in cases]
    want = [mx.rmsnorm_backward(*a) for a in dev_args]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mx.rmsnorm_backward(*dev_args[0], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    graphs, outs = [], []
    for a in dev_args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mx.rmsnorm_backward(*a))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        again = mx.rmsnorm_backward(*dev_args[1])
        torch.cuda.synchronize()
        for o, w in zip(outs + [again], want + [want[1]]):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
        for o in outs:
            o[0].zero_()
            o[1].zero_()


def test_binding_refusals(mx):
    import torch
    x = torch.zeros(4, 64, device="cuda")
    r, w = torch.ones(4, device="cuda"), torch.ones(64, device="cuda")
    for bad in (lambda: mx.rmsnorm_backward(x, x.bfloat16(), r, w),
                lambda: mx.rmsnorm_backward(x, x[:3], r, w),
                lambda: mx.rmsnorm_backward(x, x, r.double(), w),
                lambda: mx.rmsnorm_backward(x, x, r[:3], w),
                lambda: mx.rmsnorm_backward(x, x, r, w, x[:, :32]),
                lambda: mx.rmsnorm_backward(x, x, r, w, dh=x.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(mx.MxError) as e:
        mx.rmsnorm_backward(x[:, :60].contiguous(), x[:, :60].contiguous(), r, w[:60])
    assert e.value.status == -2


@pytest.mark.parametrize("rows", [0, 2])
def test_more_columns_than_a_launch_s_threads(mx, rows):
    """2^27 columns and more, 32 threads to a column in the weight gradient's
    sum: a launch may hold fewer than 2^32 threads. Sampled columns against
    fp64, with the bounds above."""
    import torch
    cols = (1 << 27) + 4104
    gen = torch.Generator(device="cuda").manual_seed(9)
    dy, h, w = (torch.randn(s, generator=gen, device="cuda").bfloat16()
                for s in ((rows, cols), (rows, cols), (cols,)))
    rstd = torch.linspace(0.5, 2.0, rows, device="cuda")
    dh, dw = mx.rmsnorm_backward(dy, h, rstd, w)
    assert dh.shape == (rows, cols) and dw.shape == (cols,)
    if rows == 0:
        assert not dw.any()
        return
    xh = h.double() * rstd.double()[:, None]
    g = dy.double() * w.double()
    m, S = (v.mean(1, keepdim=True) for v in (g * xh, (g * xh).abs()))
    pick = torch.cat([torch.arange(a, b, device="cuda") for a, b in
                      ((0, 40), ((1 << 26) - 40, (1 << 26) + 40), ((1 << 27) - 40, (1 << 27) + 40),
                       (cols - 40, cols))])
    xh, g, rs, K = xh[:, pick], g[:, pick], rstd.double()[:, None], cols / 512 + 64
    ref = rs * (g - xh * m)
    bound = rs * (6 * U * (g.abs() + (xh * m).abs()) + xh.abs() * (K + 4) * U * S) \
        + (2 * U + 2.0 ** -8) * ref.abs() + 2.0 ** -134
    assert torch.all((dh[:, pick].double() - ref).abs() <= bound)
    terms = dy[:, pick].double() * xh
    assert torch.all((dw[pick].double() - terms.sum(0)).abs() <= 69 * U * terms.abs().sum(0))


@pytest.mark.parametrize("dres", [True, False])
@pytest.mark.parametrize("rows,cols", [(16384, 4096), (2800, 12288)])
def test_rows_read_past_the_caches(mx, rows, cols, dres):
    """bf16 rows of 192 MB and more, one unit of columns to a thread and two:
    every element against fp64, with the bounds above."""
    import torch
    assert rows * cols * 2 * (4 if dres else 3) >= 192 << 20
    gen = torch.Generator(device="cuda").manual_seed(rows + dres)
    dy, h, w, d = (torch.randn(s, generator=gen, device="cuda").bfloat16()
                   for s in ((rows, cols), (rows, cols), (cols,), (rows, cols)))
    rstd = (h.double().square().mean(1) + 1e-5).rsqrt().float()
    dh, dw = mx.rmsnorm_backward(dy, h, rstd, w, d if dres else None)
    rs = rstd.double()[:, None]
    xh, g = h.double() * rs, dy.double() * w.double()
    m, S = ((g * xh).mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True))
    K = cols / 512 + 64
    ref = rs * (g - xh * m) + (d.double() if dres else 0)
    bound = rs * (6 * U * (g.abs() + (xh * m).abs()) + xh.abs() * (K + 4) * U * S) \
        + (2 * U + 2.0 ** -8) * ref.abs() + 2.0 ** -134
    if dres:
        bound += 2 * U * d.double().abs()
    assert torch.all((dh.double() - ref).abs() <= bound)
    terms = dy.double() * xh
    assert torch.all((dw.double() - terms.sum(0)).abs() <= (rows / 64 + 68) * U * terms.abs().sum(0))
