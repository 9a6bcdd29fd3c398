"""Products with an epilogue and products grouped by expert, against fp64."""
import numpy as np
import pytest

import oracle
from datagen import activations_bf16, normal_bf16
from fused_util import check, check_backward, check_forward, host64, product, values
from gpu_util import to_dev

pytestmark = pytest.mark.gpu

AXES = {"fprop": (1, 1), "dgrad": (1, 0), "wgrad": (0, 0)}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _rows(seed, shape, dtype, ld=None):
    """A random matrix; with ld a row-strided view at an odd element."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    if ld is None:
        return torch.randn(shape, generator=gen, device="cuda").to(t)
    buf = torch.randn((*shape[:-1], ld), generator=gen, device="cuda").to(t)
    return buf[..., 1:1 + shape[-1]]


def _operand(mx, rng, mn, k, axis, **how):
    shape = (mn, k) if axis == 1 else (k, mn)
    return mx.quantize(to_dev(activations_bf16(rng, shape, outlier_frac=0.01)), axis, **how)


def _pair(mx, seed, op, m, n, k):
    rng = np.random.Generator(np.random.PCG64(seed))
    qa, qb = (_operand(mx, rng, x, k, a) for x, a in zip((m, n), AXES[op]))
    return qa, qb, *product(values(qa), values(qb))


# one row to several tiles, extents that end inside one; K of one block, one slice and more
SHAPES = [(1, 1, 32), (1, 64, 128), (3, 70, 160), (16, 129, 96), (17, 65, 1056), (64, 256, 512),
          (130, 257, 288), (300, 520, 1184), (513, 300, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op", ["fprop", "dgrad", "wgrad"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(mx, shape, op, dtype):
    m, n, k = shape
    qa, qb, acc, err = _pair(mx, m + n, op, m, n, k)
    bias = _rows(1, (n,), "f32")
    mul, res = _rows(2, (m, n), dtype), _rows(3, (m, n), dtype)
    plain = mx.linear_fused(op, qa, qb, out_dtype=dtype)
    check_forward(plain, None, acc, err, dtype, "none", None, None, None, "plain")
    for i, act in enumerate(ACTS):
        b, u, r = (x if (i + j) % 3 else None for j, x in enumerate((bias, mul, res)))
        c, pre = mx.linear_fused(op, qa, qb, out_dtype=dtype, bias=b, activation=act, mul=u,
                                 residual=r, save_pre=True)
        check_forward(c, pre, acc, err, dtype, act, host64(b), host64(u), host64(r), act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(mx, shape, dtype):
    m, n, k = shape
    qa, qb, acc, err = _pair(mx, m * n, "dgrad", m, n, k)
    pre, mul = _rows(4, (m, n), dtype), _rows(5, (m, n), dtype)
    for act in ACTS:
        dz = mx.linear_act_backward(qa, qb, pre, act, out_dtype=dtype)
        check_backward(dz, None, acc, err, host64(pre), dtype, act, None, act)
        dz, dmul = mx.linear_act_backward(qa, qb, pre, act, mul=mul, out_dtype=dtype)
        check_backward(dz, dmul, acc, err, host64(pre), dtype, act, host64(mul), act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m", [5, 200])
def test_strided_and_misaligned_matrices(mx, m, dtype):
    """Row-strided views at odd addresses; what lies between the rows stays."""
    import torch
    n, k = 130, 160
    qa, qb, acc, err = _pair(mx, 9, "fprop", m, n, k)
    mul, res = _rows(6, (m, n), dtype, n + 9), _rows(7, (m, n), dtype, n + 3)
    bias = _rows(8, (n + 1,), "bf16")[1:]
    buf = torch.full((2, m, n + 5), 7.0, device="cuda").to(mul.dtype)
    out, pre = buf[0, :, 1:n + 1], buf[1, :, 3:n + 3]
    got = mx.linear_fused("fprop", qa, qb, out_dtype=dtype, bias=bias, activation="silu", mul=mul,
                          residual=res, save_pre=pre, out=out)
    assert got[0] is out and got[1] is pre
    check_forward(out, pre, acc, err, dtype, "silu", host64(bias), host64(mul), host64(res), "views")
    assert (buf[0, :, 0] == 7).all() and (buf[0, :, n + 1:] == 7).all()
    assert (buf[1, :, :3] == 7).all() and (buf[1, :, n + 3:] == 7).all()


@pytest.mark.parametrize("m", [7, 300])
def test_in_place(mx, m):
    """residual, mul and pre as the output itself."""
    n, k = 256, 128
    qa, qb, acc, err = _pair(mx, 10, "wgrad", m, n, k)
    c = _rows(11, (m, n), "f32")
    before = host64(c)
    for _ in range(2):                                 # a gradient summed over micro-batches
        mx.linear_fused("wgrad", qa, qb, out_dtype="f32", residual=c, out=c)
    check(c, before + 2 * acc, 2 * err + 2.0 ** -24 * (np.abs(before) + np.abs(before + acc)), "f32",
          "accumulated")
    g, u = _rows(12, (m, n), "bf16"), _rows(13, (m, n), "bf16")
    g0, u0 = host64(g), host64(u)
    qa, qb, acc, err = _pair(mx, 14, "dgrad", m, n, k)
    dz, dmul = mx.linear_act_backward(qa, qb, g, "silu", mul=u, out_dtype="bf16", out=g, dmul=u)
    assert dz is g and dmul is u
    check_backward(g, u, acc, err, g0, "bf16", "silu", u0, "in place")


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("rows", [8, 96])
def test_gradient_against_differences(mx, act, rows):
    """Sum of G act(z), z moved by +-h: G act'(z) within h^2 / 6 |act'''| (at most
    2) plus the two values' errors over 2 h. The products by the unit matrix hand
    G and z on exactly."""
    import torch
    rng = np.random.default_rng(rows)
    n, h = 128, 2.0 ** -7
    eye = torch.eye(n, device="cuda").bfloat16()
    q = lambda x, a: mx.quantize(x.contiguous(), a, rotate="none")  # noqa: E731
    e2m1 = np.array([.5, 1, 1.5, 2, 3, 4, 6, -.5, -1, -1.5, -2, -3, -4, -6])
    z = torch.tensor(rng.choice(e2m1, (rows, n)), device="cuda").bfloat16()
    g = torch.tensor(rng.choice(e2m1, (rows, n)), device="cuda").bfloat16()
    lo, hi = (mx.linear_fused("fprop", q(z, 1), q(eye, 1), activation=act,
                              bias=torch.full((n,), s * h, device="cuda")) for s in (-1, 1))
    diff = g.double() * (hi.double() - lo.double()) / (2 * h)
    dz = mx.linear_act_backward(q(g, 1), q(eye, 0), z.float(), act)
    bound = g.double().abs() * (h * h / 3 + 2.0 ** -20 * (1 + z.double().abs() + h) / h + 2.0 ** -18)
    assert ((dz.double() - diff).abs() <= bound).all()


@pytest.mark.parametrize("m", [3, 300])
def test_special_values(mx, m):
    """Infinities in the epilogue's inputs: the activations' limits; NaN stays."""
    import torch
    n, k = 64, 32
    qa, qb, acc, err = _pair(mx, 15, "fprop", m, n, k)
    qg, qw, gacc, gerr = _pair(mx, 15, "dgrad", m, n, k)
    bias = torch.zeros(n, device="cuda")
    bias[3], bias[10], bias[20], bias[30], bias[40] = (float("inf"), float("-inf"), float("nan"),
                                                       1e30, -1e30)
    for act in ACTS:
        c = mx.linear_fused("fprop", qa, qb, bias=bias, activation=act)
        assert (c[:, 3] == float("inf")).all() and c[:, 20].isnan().all(), act
        low = float("-inf") if act == "none" else 0.0
        assert (c[:, 10] == low).all(), act
        assert (c[:, 30] == 1e30).all() and (c[:, 40] == (-1e30 if act == "none" else 0)).all(), act
        rest = np.array([i for i in range(n) if i not in (3, 10, 20, 30, 40)])
        check_forward(c[:, rest], None, acc[:, rest], err[:, rest], "f32", act, None, None, None, act)
        pre = bias.expand(m, n).contiguous()
        dz = mx.linear_act_backward(qg, qw, pre, act)
        want = 1.0 if act == "none" else 0.0
        for col, slope in ((3, 1.0), (10, want), (30, 1.0), (40, want)):
            check(dz[:, col], gacc[:, col] * slope, gerr[:, col], "f32", act)
        assert act in ("none", "relu") or dz[:, 20].isnan().all()


def test_no_reduction(mx):
    """K == 0: the sums are zeros."""
    import torch
    a = mx.quantize(torch.empty((5, 0), dtype=torch.bfloat16, device="cuda"), 1)
    b = mx.quantize(torch.empty((40, 0), dtype=torch.bfloat16, device="cuda"), 1)
    bias = _rows(16, (40,), "f32")
    c = mx.linear_fused("fprop", a, b, bias=bias, activation="relu")
    assert torch.equal(c, bias.clamp(min=0).expand(5, 40))
    assert mx.linear_fused("fprop", mx.quantize(torch.empty((0, 32), dtype=torch.bfloat16,
                                                            device="cuda"), 1),
                           mx.quantize(torch.ones((4, 32), device="cuda").bfloat16(), 1)).shape == (0, 4)


# ---- grouped ----------------------------------------------------------------

def _grouped(mx, seed, sizes, spare, out, cin, **how):
    """Rows [T, in], [T, out] and stacked matrices [E, out, in], quantized."""
    import torch
    rng = np.random.Generator(np.random.PCG64(seed))
    t, e = sum(sizes) + spare, len(sizes)
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    x, dy = (to_dev(activations_bf16(rng, (t, c), outlier_frac=0.01)) for c in (cin, out))
    w = to_dev(normal_bf16(rng, (e * out, cin), 0.05)).view(e, out, cin)
    return (ends, mx.quantize_grouped(x, ends, **how), mx.quantize_grouped(dy, ends, **how),
            mx.quantize_grouped(w, **how))


def _grouped_ref(op, qa, qb, ranges, out, cin):
    """[(place in C, acc, bound)] of the groups."""
    a, b = values(qa), values(qb)
    kp, at, found = -(-out // 128) * 128, 0, []
    for e, (first, last) in enumerate(ranges):
        deep = -(-(last - first) // 128) * 128
        if op == "fprop":
            part = slice(first, last), a[first:last], b[e * out:(e + 1) * out]
        elif op == "dgrad":
            part = slice(first, last), a[first:last], b[:, e * kp:e * kp + out]
        else:
            part = e, a[:, at:at + deep], b[:, at:at + deep]
        found.append((part[0], *product(part[1], part[2])))
        at += deep
    return found


GROUPS = [([1], 0, 64, 32), ([5], 3, 96, 64), ([3, 0, 1, 12], 0, 128, 160), ([0, 0, 9], 2, 33, 96),
          ([40, 7, 0, 100, 64, 65], 9, 160, 288), ([300, 0, 5, 213], 20, 320, 96),
          ([1] * 70, 1, 64, 64), ([0, 0], 6, 64, 32), ([700, 129], 0, 257, 512)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,spare,out,cin", GROUPS)
@pytest.mark.parametrize("op", ["fprop", "dgrad", "wgrad"])
def test_grouped(mx, op, sizes, spare, out, cin, dtype):
    import torch
    if op == "dgrad":
        out = -(-out // 32) * 32                       # dY's blocks run along `out`
    if op == "wgrad":
        out, cin = -(-out // 32) * 32, cin
    how = {} if out % 32 == 0 else None
    if how is None:                                    # fprop with an odd number of outputs
        rng = np.random.Generator(np.random.PCG64(1))
        e = len(sizes)
        ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
        x = to_dev(activations_bf16(rng, (sum(sizes) + spare, cin), outlier_frac=0.01))
        w = to_dev(normal_bf16(rng, (e * out, cin), 0.05)).view(e, out, cin)
        qa, qb = mx.quantize_grouped(x, ends, dual=False).q1, mx.quantize_grouped(w).q1
    else:
        ends, x, dy, w = _grouped(mx, len(sizes) + out, sizes, spare, out, cin)
        qa, qb = {"fprop": (x.q1, w.q1), "dgrad": (dy.q1, w.q0), "wgrad": (dy.q0, x.q0)}[op]
    t, e = sum(sizes) + spare, len(sizes)
    shape = (e, out, cin) if op == "wgrad" else (t, out if op == "fprop" else cin)
    ref = _grouped_ref(op, qa, qb, oracle.group_ranges_ref(np.cumsum(sizes), t), out, cin)
    bias = _rows(21, (e, shape[-1]), "f32")
    mul, res = _rows(22, shape, dtype), _rows(23, shape, dtype)
    for b, act, u, r in ((None, "none", None, None), (bias, "silu", mul, None),
                         (bias, "gelu_tanh", None, res)):
        c, pre = torch.full((2, *shape), 3.0, device="cuda").to(res.dtype)
        mx.linear_grouped(op, qa, qb, ends, out_dtype=dtype, bias=b, activation=act, mul=u,
                          residual=r, save_pre=pre, out=c)
        for i, (at, acc, err) in enumerate(ref):
            pick = lambda v: None if v is None else host64(v)[at]  # noqa: E731
            check_forward(c[at], pre[at], acc, err, dtype, act, None if b is None else host64(b)[i],
                          pick(u), pick(r), f"group {i}")
        if op != "wgrad":                              # rows behind the last end
            assert (c[sum(sizes):] == 3).all() and (pre[sum(sizes):] == 3).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,spare,out,cin", [([1], 0, 64, 64), ([3, 0, 30], 4, 96, 160),
                                                 ([260, 1, 90], 7, 288, 320)])
def test_grouped_backward(mx, sizes, spare, out, cin, dtype):
    import torch
    ends, _, dy, w = _grouped(mx, 31, sizes, spare, out, cin)
    t = sum(sizes) + spare
    ref = _grouped_ref("dgrad", dy.q1, w.q0, oracle.group_ranges_ref(np.cumsum(sizes), t), out, cin)
    pre, mul = _rows(32, (t, cin), dtype), _rows(33, (t, cin), dtype)
    c, d = torch.full((2, t, cin), 3.0, device="cuda").to(pre.dtype)
    mx.linear_act_backward(dy.q1, w.q0, pre, "gelu", mul=mul, ends=ends, out_dtype=dtype, out=c,
                           dmul=d)
    for at, acc, err in ref:
        check_backward(c[at], d[at], acc, err, host64(pre)[at], dtype, "gelu", host64(mul)[at], "")
    assert (c[sum(sizes):] == 3).all() and (d[sum(sizes):] == 3).all()


@pytest.mark.parametrize("rotate,rnd", [("rand_sign_hadamard", "sr"), ("hadamard16", "rne"),
                                        ("none", "sr")])
@pytest.mark.parametrize("op", ["fprop", "dgrad", "wgrad"])
def test_grouped_rotations_cancel(mx, op, rotate, rnd):
    """The product of the packed values is near the product of the sources: the
    two operands' signs belong together."""
    import torch
    rng = np.random.Generator(np.random.PCG64(41))
    sizes, out, cin = [150, 0, 77], 96, 128
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    x, dy = (to_dev(normal_bf16(rng, (227, c), 1.0)) for c in (cin, out))
    w = to_dev(normal_bf16(rng, (3 * out, cin), 1.0)).view(3, out, cin)
    how = {"rotate": rotate, "round": rnd, "seed1": 6, "seed0": 6 | 1 << 32}
    qx, qdy, qw = (mx.quantize_grouped(x, ends, **how), mx.quantize_grouped(dy, ends, **how),
                   mx.quantize_grouped(w, **how))
    qa, qb = {"fprop": (qx.q1, qw.q1), "dgrad": (qdy.q1, qw.q0), "wgrad": (qdy.q0, qx.q0)}[op]
    got = host64(mx.linear_grouped(op, qa, qb, ends))
    xs, ds, ws = host64(x), host64(dy), host64(w)
    for e, (a, b) in enumerate(oracle.group_ranges_ref(np.cumsum(sizes), 227)):
        ref = {"fprop": xs[a:b] @ ws[e].T, "dgrad": ds[a:b] @ ws[e], "wgrad": ds[a:b].T @ xs[a:b]}[op]
        mine = got[e] if op == "wgrad" else got[a:b]
        # two operands of about 12% (nearest) to 16% (stochastic) quantization noise
        assert b == a or np.linalg.norm(mine - ref) < 0.3 * np.linalg.norm(ref)
        assert b > a or not mine.any()


def test_nan_reaches_its_own_group_only(mx):
    import torch
    rng = np.random.Generator(np.random.PCG64(51))
    sizes, out, cin = [37, 40, 3], 96, 64
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    x = to_dev(normal_bf16(rng, (90, cin), 1.0))
    dy = to_dev(normal_bf16(rng, (90, out), 1.0))
    w = to_dev(normal_bf16(rng, (3 * out, cin), 1.0)).view(3, out, cin)
    x[38, 5], w[2, 7, 9], x[85] = float("nan"), float("inf"), float("nan")
    qx, qdy, qw = mx.quantize_grouped(x, ends), mx.quantize_grouped(dy, ends), mx.quantize_grouped(w)
    y = mx.linear_grouped("fprop", qx.q1, qw.q1, ends)[:80].isnan()
    want = torch.zeros_like(y)
    want[38], want[77:80, 7] = True, True
    assert torch.equal(y, want)
    d = mx.linear_grouped("dgrad", qdy.q1, qw.q0, ends)[:80].isnan()
    want = torch.zeros_like(d)
    want[77:80, 9] = True
    assert torch.equal(d, want)
    g = mx.linear_grouped("wgrad", qdy.q0, qx.q0, ends).isnan()
    want = torch.zeros_like(g)
    want[1, :, 5] = True
    assert torch.equal(g, want)


def test_an_ordinary_operand_as_rows(mx):
    """A of the forward product from quantize and rmsnorm_quantize; ends that
    only the device knows and that change between the calls."""
    import torch
    rng = np.random.Generator(np.random.PCG64(61))
    x = to_dev(normal_bf16(rng, (100, 128), 1.0))
    w = to_dev(normal_bf16(rng, (2 * 64, 128), 0.1)).view(2, 64, 128)
    qw = mx.quantize_grouped(w)
    ends = torch.zeros(2, dtype=torch.int32, device="cuda")
    for a in (mx.quantize(x, 1), mx.rmsnorm_quantize(x, torch.ones(128, device="cuda")).q1):
        for split in (0, 33, 64, 100):
            ends.copy_(torch.tensor([split, 100]))
            c = mx.linear_grouped("fprop", a, qw.q1, ends)
            acc, err = product(values(a), values(qw.q1))
            check(c[:split], acc[:split, :64], err[:split, :64], "f32", "first")
            check(c[split:], acc[split:, 64:], err[split:, 64:], "f32", "second")
