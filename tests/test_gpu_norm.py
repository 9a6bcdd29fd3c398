"""RMS norm into packed operands on the GPU against the oracle: h, rstd, codes
and scales bit for bit.

rstd is rounded once from a 64-bit sum, so the order of the sum can change it
only where the exact value lies within about 1e-15 of a rounding border of
fp32 (2^-24 apart): about one row in 10^7, none at these seeds.
"""
import numpy as np
import pytest

import oracle
from norm_util import check_operand, dev, host, values

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _case(mx, rows, cols, bf16=True, wbf16=True, residual=True, dual=False, fmt="fp8_e4m3",
          rotate="hadamard", rnd="rne", seed=3, eps=EPS, ld=None, x=None, r=None, w=None):
    rng = np.random.default_rng(rows * 131 + cols)
    x = values(rng, (rows, cols), bf16) if x is None else x
    if r is None and residual:
        r = values(rng, (rows, cols), bf16)
    w = values(rng, (cols,), wbf16) if w is None else w
    h, rstd, y = oracle.rmsnorm_ref(x, w, r, eps, bf16)
    seed0 = seed | 1 << 32
    got = mx.rmsnorm_quantize(dev(x, bf16, ld), dev(w, wbf16),
                              None if r is None else dev(r, bf16, ld), eps=eps, format=fmt,
                              dual=dual, rotate=rotate, round=rnd, seed1=seed, seed0=seed0)
    what = f"{rows}x{cols} {fmt} {rotate} {rnd}"
    assert np.array_equal(host(got.h), h, equal_nan=True), what + " h"
    assert np.array_equal(host(got.rstd), rstd, equal_nan=True), what + " rstd"
    check_operand(got.q1, y, 1, rotate, rnd, seed, fmt, what + " axis 1")
    if dual:
        check_operand(got.q0, y, 0, rotate, rnd, seed0, fmt, what + " axis 0")
    else:
        assert got.q0 is None
    return got


SHAPES = [(1, 32), (1, 128), (1, 4096), (2, 160), (16, 128), (17, 2080), (15, 96), (255, 96),
          (257, 416), (300, 1056), (33, 14336), (5, 16416), (64, 8192)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("bf16", [True, False])
def test_axis1_shapes(mx, rows, cols, bf16):
    _case(mx, rows, cols, bf16=bf16, wbf16=not bf16)
    _case(mx, rows, cols, bf16=bf16, residual=False, fmt="fp4_e2m1", rotate="none")


@pytest.mark.parametrize("rows,cols", [(32, 32), (32, 4096), (64, 96), (96, 2080), (288, 416),
                                       (1024, 256), (32, 16416), (160, 5152)])
@pytest.mark.parametrize("bf16", [True, False])
def test_dual_shapes(mx, rows, cols, bf16):
    _case(mx, rows, cols, bf16=bf16, dual=True)
    _case(mx, rows, cols, bf16=bf16, wbf16=False, residual=False, dual=True, fmt="fp4_e2m1",
          rotate="hadamard16")


@pytest.mark.parametrize("dual", [False, True])
@pytest.mark.parametrize("rotate", ["none", "hadamard", "rand_sign_hadamard", "hadamard16"])
@pytest.mark.parametrize("fmt,rnd", [("fp4_e2m1", "rne"), ("fp4_e2m1", "sr"), ("fp8_e4m3", "rne")])
def test_every_variant(mx, fmt, rnd, rotate, dual):
    for bf16 in (True, False):
        _case(mx, 96, 288, bf16=bf16, fmt=fmt, rnd=rnd, rotate=rotate, dual=dual, seed=11)
        _case(mx, 32, 4128, bf16=bf16, fmt=fmt, rnd=rnd, rotate=rotate, dual=dual, seed=12)


def _special(rows, cols, bf16, rng):
    """Rows of zeros, of one spike, of huge and of tiny values, with a NaN, with
    infinities, and infinities of both signs."""
    x = values(rng, (rows, cols), bf16)
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 0.0
    x[2, 5] = 1.0
    x[3] *= np.float32(2.0 ** 100)             # squares beyond fp32
    x[4] *= np.float32(2.0 ** -120)            # squares below it; some values subnormal
    x[5, 40] = np.nan
    x[6, 7] = np.inf
    x[7, 9], x[7, 70] = -np.inf, np.inf
    x[8] = np.float32(2.0 ** -133)             # bf16's smallest
    return x


@pytest.mark.parametrize("dual", [False, True])
@pytest.mark.parametrize("rotate", ["none", "hadamard", "hadamard16"])
@pytest.mark.parametrize("bf16", [True, False])
def test_special_rows(mx, bf16, rotate, dual):
    x = _special(32, 160, bf16, np.random.default_rng(7))
    w = np.abs(values(np.random.default_rng(8), (160,), True)) + np.float32(0.5)
    w = dev(w, True).float().cpu().numpy()
    for fmt in ("fp4_e2m1", "fp8_e4m3"):
        for eps in (EPS, 0.0):
            _case(mx, 32, 160, bf16=bf16, residual=False, dual=dual, fmt=fmt, rotate=rotate,
                  eps=eps, x=x, w=w)
    r = np.zeros_like(x)
    r[6, 7] = -np.inf                          # inf - inf in the stream
    _case(mx, 32, 160, bf16=bf16, dual=dual, rotate=rotate, x=x, r=r, w=w)


def test_strided_rows_and_untouched_padding(mx):
    """Row-strided sources with NaN padding; h written through a row-strided
    view of a larger buffer leaves everything around it alone."""
    import torch
    _case(mx, 37, 224, ld=240)
    _case(mx, 64, 224, ld=228, bf16=False, dual=True)
    rng = np.random.default_rng(9)
    x, r, w = values(rng, (20, 96), True), values(rng, (20, 96), True), values(rng, (96,), True)
    big = torch.full((33, 120), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mx.rmsnorm_quantize(dev(x, True), dev(w, True), dev(r, True), h=big[3:23, 8:104],
                              format="fp8_e4m3")
    h, _, y = oracle.rmsnorm_ref(x, w, r, EPS, True)
    assert np.array_equal(host(big[3:23, 8:104]), h)
    big[3:23, 8:104] = 7.0
    assert torch.all(big == 7.0)
    check_operand(got.q1, y, 1, "hadamard", "rne", 0, "fp8_e4m3", "strided h")


@pytest.mark.parametrize("cols", [96, 4096, 16416])
@pytest.mark.parametrize("bf16", [True, False])
def test_in_place(mx, cols, bf16):
    """The stream updated in place, over residual or over x."""
    rng = np.random.default_rng(10)
    x, r, w = (values(rng, (32, cols), bf16), values(rng, (32, cols), bf16),
               values(rng, (cols,), True))
    h, _, y = oracle.rmsnorm_ref(x, w, r, EPS, bf16)
    for dual in (False, True):
        for over in ("x", "residual"):
            tx, tr = dev(x, bf16), dev(r, bf16)
            t = tx if over == "x" else tr
            got = mx.rmsnorm_quantize(tx, dev(w, True), tr, h=t, dual=dual, format="fp8_e4m3")
            assert got.h is t and np.array_equal(host(t), h)
            check_operand(got.q1, y, 1, "hadamard", "rne", 0, "fp8_e4m3", over)
            if dual:
                check_operand(got.q0, y, 0, "hadamard", "rne", 0, "fp8_e4m3", over)


def test_large_rows_sampled(mx):
    """The block's tokens and width, where the rows outgrow the caches: the
    first, middle and last row blocks against the oracle."""
    import torch
    rows, cols = 16384, 4096
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(rows, cols, generator=gen, device="cuda").bfloat16()
    r = torch.randn(rows, cols, generator=gen, device="cuda").bfloat16()
    w = 1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")
    _sampled(mx, x, w, r, np.r_[0:32, 8160:8224, 16352:16384], True)
    _sampled(mx, x, w, r, np.r_[0:32, 8160:8224, 16352:16384], False)


def _sampled(mx, x, w, r, pick, dual, fmt="fp8_e4m3", bf16=True):
    """Rows `pick` (whole 32-row blocks with dual) against the oracle."""
    rows, cols = x.shape
    got = mx.rmsnorm_quantize(x, w, r, dual=dual, format=fmt)
    h, rstd, y = oracle.rmsnorm_ref(host(x[pick]), host(w), host(r[pick]), EPS, bf16)
    assert np.array_equal(host(got.h[pick]), h) and np.array_equal(host(got.rstd[pick]), rstd)
    q = oracle.quantize_values_ref(y, 1, fmt=fmt)
    codes, scales = got.q1.codes.cpu().numpy(), got.q1.scales.cpu().numpy()
    assert np.array_equal(oracle.untile_codes_fp8(codes, rows, cols)[pick], q.codes)
    assert np.array_equal(oracle.untile_scales(scales, rows, cols)[pick], q.scales)
    if dual:
        q = oracle.quantize_values_ref(y, 0, fmt=fmt)
        codes, scales = got.q0.codes.cpu().numpy(), got.q0.scales.cpu().numpy()
        blocks = pick.reshape(-1, 32)[:, 0] // 32
        assert np.array_equal(oracle.untile_codes_fp8(codes, cols, rows)[:, pick], q.codes)
        assert np.array_equal(oracle.untile_scales(scales, cols, rows)[:, blocks], q.scales)


def test_large_f32_rows_sampled(mx):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, r = (torch.randn(4096, 4096, generator=gen, device="cuda") for _ in range(2))
    w = (1 + 0.1 * torch.randn(4096, generator=gen, device="cuda")).bfloat16()
    for dual in (False, True):
        _sampled(mx, x, w, r, np.r_[0:32, 2016:2080, 4064:4096], dual, bf16=False)


def test_many_rows(mx):
    """More 32-row pieces than a grid's second extent may count (65535)."""
    import torch
    rows, cols = 65536 * 32 + 64, 32
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, r = (torch.randn(rows, cols, generator=gen, device="cuda").bfloat16() for _ in range(2))
    w = 1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")
    pick = np.r_[0:32, 65535 * 32:65537 * 32, rows - 32:rows]
    _sampled(mx, x, w, r, pick, True)


@pytest.mark.parametrize("dual", [False, True])
def test_offsets_beyond_32_bits(mx, dual):
    """Rows that lie more than 4 GiB after the first."""
    import torch
    rows, cols, ld = 64, 256, 1 << 26
    big = torch.empty((rows * ld,), dtype=torch.bfloat16, device="cuda").view(rows, ld)
    x = big[:, 64:64 + cols]
    r, h = big[:, 1024:1024 + cols], big[:, 4096:4096 + cols]
    rng = np.random.default_rng(15)
    xv, rv, w = (values(rng, s, True) for s in ((rows, cols), (rows, cols), (cols,)))
    x.copy_(dev(xv, True))
    r.copy_(dev(rv, True))
    got = mx.rmsnorm_quantize(x, dev(w, True), r, h=h, dual=dual, format="fp8_e4m3")
    href, rstd, y = oracle.rmsnorm_ref(xv, w, rv, EPS, True)
    assert np.array_equal(host(h), href) and np.array_equal(host(got.rstd), rstd)
    check_operand(got.q1, y, 1, "hadamard", "rne", 0, "fp8_e4m3", "far rows")
    if dual:
        check_operand(got.q0, y, 0, "hadamard", "rne", 0, "fp8_e4m3", "far rows")


def test_operand_feeds_linear(mx):
    """The operand goes into the linear as a quantized one does."""
    rng = np.random.default_rng(12)
    x, r, w = values(rng, (70, 256), True), values(rng, (70, 256), True), values(rng, (256,), True)
    W = values(rng, (96, 256), True, 0.02)
    _, _, y = oracle.rmsnorm_ref(x, w, r, EPS, True)
    for fmt, quant in (("fp4_e2m1", mx.quantize), ("fp8_e4m3", mx.quantize_fp8)):
        q = mx.rmsnorm_quantize(dev(x, True), dev(w, True), dev(r, True), format=fmt).q1
        c = host(mx.linear("fprop", q, quant(dev(W, True), 1)))
        qa = oracle.quantize_values_ref(y, 1, fmt=fmt)
        qb = oracle.quantize_values_ref(W, 1, fmt=fmt)
        ref = oracle.mx_gemm_ref(qa, qb)
        err = np.linalg.norm(c - ref) / np.linalg.norm(ref)
        # MXFP4 accumulates exactly per block (1e-5); E4M3's matrix instruction
        # drops product bits below 2^-13 of a block's largest (1e-4)
        assert err <= (1e-5 if fmt == "fp4_e2m1" else 1e-4), (fmt, err)


def test_empty(mx):
    import torch
    for rows, cols in ((0, 64), (32, 0)):
        x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        w = torch.ones(cols, device="cuda")
        got = mx.rmsnorm_quantize(x, w, x.clone(), dual=True)
        assert got.q1.codes.numel() == 0 and got.q0.source_shape == (rows, cols)
        assert got.rstd.shape == (rows,)


def test_another_stream(mx):
    import torch
    rng = np.random.default_rng(13)
    x, r, w = values(rng, (96, 512), True), values(rng, (96, 512), True), values(rng, (512,), True)
    h, _, y = oracle.rmsnorm_ref(x, w, r, EPS, True)
    tx, tr, tw = dev(x, True), dev(r, True), dev(w, True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, torch.cuda.current_stream().cuda_stream):
        got = mx.rmsnorm_quantize(tx, tw, tr, dual=True, format="fp8_e4m3", stream=stream)
        torch.cuda.synchronize()
        check_operand(got.q1, y, 1, "hadamard", "rne", 0, "fp8_e4m3", "stream")
        check_operand(got.q0, y, 0, "hadamard", "rne", 0, "fp8_e4m3", "stream")


@pytest.mark.parametrize("dual", [False, True])
def test_captured_and_replayed(mx, dual):
    """A captured call replayed on new inputs, with eager work in between,
    gives the eager call's bytes every time."""
    import torch
    rng = np.random.default_rng(14)
    shape = (64, 1056)
    x, r, w = dev(values(rng, shape, True), True), dev(values(rng, shape, True), True), \
        dev(values(rng, (1056,), True), True)
    mx.rmsnorm_quantize(x, w, r, dual=dual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mx.rmsnorm_quantize(x, w, r, dual=dual)
    for _ in range(4):
        x.copy_(dev(values(rng, shape, True), True))
        r.copy_(dev(values(rng, shape, True), True))
        want = mx.rmsnorm_quantize(x, w, r, dual=dual)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.h, want.h) and torch.equal(got.rstd, want.rstd)
        assert torch.equal(got.q1.codes, want.q1.codes)
        assert torch.equal(got.q1.scales, want.q1.scales)
        if dual:
            assert torch.equal(got.q0.codes, want.q0.codes)
            assert torch.equal(got.q0.scales, want.q0.scales)


def test_binding_refusals(mx):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (lambda: mx.rmsnorm_quantize(x.half(), w),
                lambda: mx.rmsnorm_quantize(x, w.half()),
                lambda: mx.rmsnorm_quantize(x, w[:32]),
                lambda: mx.rmsnorm_quantize(x, w, x.float()),
                lambda: mx.rmsnorm_quantize(x, w, x[:2]),
                lambda: mx.rmsnorm_quantize(x.t(), w[:4]),
                lambda: mx.rmsnorm_quantize(x, w, h=x.clone()),
                lambda: mx.rmsnorm_quantize(x, w, x.clone(), h=x.float()),
                lambda: mx.rmsnorm_quantize(x, torch.ones(128, device="cuda")[::2])):
        with pytest.raises(ValueError):
            bad()
    for status, bad in ((-4, lambda: mx.rmsnorm_quantize(x, w, format="fp8_e4m3", round="sr")),
                        (-2, lambda: mx.rmsnorm_quantize(x, w, dual=True)),
                        (-3, lambda: mx.rmsnorm_quantize(x, torch.ones(65, device="cuda")[1:])),
                        (-4, lambda: mx.rmsnorm_quantize(x, w, eps=-1.0))):
        with pytest.raises(mx.MxError) as e:
            bad()
        assert e.value.status == status


@pytest.mark.parametrize("rows,cols", [(8192, 4096), (4096, 8224)])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("fmt,rnd,rotate", [("fp4_e2m1", "rne", "hadamard"),
                                            ("fp4_e2m1", "sr", "rand_sign_hadamard"),
                                            ("fp8_e4m3", "rne", "hadamard16")])
def test_rows_read_past_the_caches(mx, fmt, rnd, rotate, bf16, rows, cols):
    """Rows of 192 MB and more take kernels that read and write around the
    caches: the first 512 rows come out as those rows alone do (checked against
    the oracle at such sizes above). Tiles of 16 rows follow each other in the
    axis-1 operand; in the axis-0 one the first 512 rows are the first K."""
    import torch
    some = 512
    assert rows * cols * (2 if bf16 else 4) * 3 >= 192 << 20 > some * cols * 4 * 3
    gen = torch.Generator(device="cuda").manual_seed(8)
    x, r = (torch.randn(rows, cols, generator=gen, device="cuda") for _ in range(2))
    x, r = (x.bfloat16(), r.bfloat16()) if bf16 else (x, r)
    w = 1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")
    for dual in (False, True):
        kw = dict(format=fmt, rotate=rotate, round=rnd, seed1=5, seed0=6 | 1 << 32, dual=dual)
        got = mx.rmsnorm_quantize(x, w, r, **kw)
        want = mx.rmsnorm_quantize(x[:some], w, r[:some], **kw)
        assert torch.equal(got.h, x + r) and torch.equal(got.rstd[:some], want.rstd)
        n = want.q1.codes.numel()
        assert torch.equal(got.q1.codes[:n], want.q1.codes)
        shape = -1, 1024                        # scales: [K / 128][MN / 256][1024]
        a, b = (q.q1.scales.view(-(-cols // 128), *shape) for q in (got, want))
        assert torch.equal(a[:, :some // 256], b)
        if dual:
            tile = 2048 if fmt == "fp8_e4m3" else 1024    # [MN / 16][K / 128][tile]
            a, b = (q.q0.codes.view(-1, k // 128, tile) for q, k in ((got, rows), (want, some)))
            assert torch.equal(a[:, :some // 128], b)
            a, b = (q.q0.scales.view(k // 128, -1) for q, k in ((got, rows), (want, some)))
            assert torch.equal(a[:some // 128], b)
