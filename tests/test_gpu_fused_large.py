"""Products with an epilogue and grouped ones, of sizes with enough 64x64 tiles
(more than three a compute unit, and columns in multiples of 64 or more than 160
GFLOP) for the kernel of 256x256 tiles, and beside those limits: tiles cut by the
matrix's ends, halves of tiles, several tiles a workgroup, matrices read and
written by columns, groups that end inside a tile. Against fp64."""
import numpy as np
import pytest

import oracle
from datagen import activations_bf16, normal_bf16
from fused_util import check, check_backward, check_forward, host64, product, values
from gpu_util import to_dev
from test_gpu_fused import _grouped_ref, _pair, _rows

pytestmark = pytest.mark.gpu

# N of whole 16-byte units, of 4-element ones only (fp32: whole, bf16: not), odd
SHAPES = [(1100, 3136, 160), (1290, 3204, 96), (1100, 3905, 288), (1290, 3200, 96), (1100, 3904, 288)]
WAYS = [("none", "b"), ("relu", "bm"), ("silu", "br"), ("gelu", "mr"), ("gelu_tanh", "bmr"),
        ("silu", "m"), ("none", "r"), ("gelu", "")]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,op", zip(SHAPES, ["fprop", "dgrad", "wgrad", "dgrad", "wgrad"]))
def test_forward(mx, shape, op, dtype):
    m, n, k = shape
    qa, qb, acc, err = _pair(mx, m + n, op, m, n, k)
    bias, mul, res = _rows(1, (n,), "f32"), _rows(2, (m, n), dtype), _rows(3, (m, n), dtype)
    for i, (act, what) in enumerate(WAYS):
        b, u, r = (x if c in what else None for c, x in zip("bmr", (bias, mul, res)))
        got = mx.linear_fused(op, qa, qb, out_dtype=dtype, bias=b, activation=act, mul=u,
                              residual=r, save_pre=i % 2 == 0)
        c, pre = got if i % 2 == 0 else (got, None)
        check_forward(c, pre, acc, err, dtype, act, host64(b), host64(u), host64(r), f"{act} {what}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(mx, shape, dtype):
    import torch
    m, n, k = shape
    qa, qb, acc, err = _pair(mx, m * n, "dgrad", m, n, k)
    pre, mul = _rows(4, (m, n), dtype), _rows(5, (m, n), dtype)
    for i, act in enumerate(("none", "relu", "silu", "gelu", "gelu_tanh")):
        u = mul if i % 2 else None
        got = mx.linear_act_backward(qa, qb, pre, act, mul=u, out_dtype=dtype)
        dz, dmul = got if u is not None else (got, None)
        check_backward(dz, dmul, acc, err, host64(pre), dtype, act, host64(u), act)
    dz, dmul = mx.linear_act_backward(qa, qb, pre, "silu", mul=mul, out_dtype=dtype, out=pre, dmul=mul)
    assert torch.equal(dz, mx.linear_act_backward(qa, qb, _rows(4, (m, n), dtype), "silu",
                                                  mul=_rows(5, (m, n), dtype), out_dtype=dtype)[0])


@pytest.mark.parametrize("op,act", [("fprop", "silu"), ("wgrad", "gelu")])
def test_several_tiles_a_workgroup(mx, op, act):
    """More than 256 tiles of 256x256, the last round of them cut in halves."""
    m, n, k = 4200, 4352, 64
    qa, qb, acc, err = _pair(mx, 3, op, m, n, k)
    mul = _rows(2, (m, n), "bf16")
    c, pre = mx.linear_fused(op, qa, qb, out_dtype="bf16", activation=act, mul=mul, save_pre=True)
    check_forward(c, pre, acc, err, "bf16", act, None, host64(mul), None, "large")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [3600, 3648])
def test_strided_and_misaligned_matrices(mx, n, dtype):
    """Row-strided views at odd addresses; what lies between the rows stays."""
    import torch
    m, k = 1250, 160
    qa, qb, acc, err = _pair(mx, 9, "fprop", m, n, k)
    mul, res = _rows(6, (m, n), dtype, n + 9), _rows(7, (m, n), dtype, n + 3)
    bias = _rows(8, (n + 1,), "bf16")[1:]
    buf = torch.full((2, m, n + 5), 7.0, device="cuda").to(mul.dtype)
    out, pre = buf[0, :, 1:n + 1], buf[1, :, 3:n + 3]
    mx.linear_fused("fprop", qa, qb, out_dtype=dtype, bias=bias, activation="silu", mul=mul,
                    residual=res, save_pre=pre, out=out)
    check_forward(out, pre, acc, err, dtype, "silu", host64(bias), host64(mul), host64(res), "views")
    assert (buf[0, :, 0] == 7).all() and (buf[0, :, n + 1:] == 7).all()
    assert (buf[1, :, :3] == 7).all() and (buf[1, :, n + 3:] == 7).all()
    # aligned rows with a space behind them: read and written in whole units
    wide = torch.full((m, n + 64), 7.0, device="cuda").to(mul.dtype)
    mx.linear_fused("fprop", qa, qb, out_dtype=dtype, activation="relu", out=wide[:, :n])
    check_forward(wide[:, :n], None, acc, err, dtype, "relu", None, None, None, "aligned view")
    assert (wide[:, n:] == 7).all()


def test_accumulated_in_place(mx):
    m, n, k = 1100, 3136, 288
    qa, qb, acc, err = _pair(mx, 10, "wgrad", m, n, k)
    c = _rows(11, (m, n), "f32")
    before = host64(c)
    for _ in range(2):
        mx.linear_fused("wgrad", qa, qb, out_dtype="f32", residual=c, out=c)
    check(c, before + 2 * acc, 2 * err + 2.0 ** -24 * (np.abs(before) + np.abs(before + acc)), "f32",
          "accumulated")


def test_special_values(mx):
    """Infinities and NaN in the epilogue's inputs stay in their columns."""
    import torch
    m, n, k = 1030, 3200, 64
    qa, qb, acc, err = _pair(mx, 15, "fprop", m, n, k)
    qg, qw, gacc, gerr = _pair(mx, 15, "dgrad", m, n, k)
    bias = torch.zeros(n, device="cuda")
    where = [3, 1010, 2020, 3030, 3199]
    bias[where] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1e30, -1e30], device="cuda")
    rest = np.setdiff1d(np.arange(n), where)
    for act in ("none", "relu", "silu", "gelu", "gelu_tanh"):
        c = mx.linear_fused("fprop", qa, qb, bias=bias, activation=act)
        low = float("-inf") if act == "none" else 0.0
        assert (c[:, 3] == float("inf")).all() and (c[:, 1010] == low).all(), act
        assert c[:, 2020].isnan().all() and (c[:, 3030] == 1e30).all(), act
        assert (c[:, 3199] == (-1e30 if act == "none" else 0)).all(), act
        check_forward(c[:, rest], None, acc[:, rest], err[:, rest], "f32", act, None, None, None, act)
        dz = mx.linear_act_backward(qg, qw, bias.expand(m, n).contiguous(), act)
        flat = 1.0 if act == "none" else 0.0
        for col, slope in ((3, 1.0), (1010, flat), (3030, 1.0), (3199, flat)):
            check(dz[:, col], gacc[:, col] * slope, gerr[:, col], "f32", act)
        assert act in ("none", "relu") or dz[:, 2020].isnan().all()


def test_ends_inside_a_tile(mx):
    """More than 160 GFLOP: the tile kernel's last columns, odd rows apart."""
    import torch
    m, n, k = 4224, 4331, 4608
    gen = torch.Generator(device="cuda").manual_seed(3)
    new = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    qa, qb, qw = mx.quantize(new(m, k), 1), mx.quantize(new(n, k), 1), mx.quantize(new(k, n), 0)
    va, vb, vw = (torch.tensor(values(q), device="cuda") for q in (qa, qb, qw))

    def exact(v):
        return ((va @ v.T).cpu().numpy(),
                ((k / 128 + 10) * 2.0 ** -22 * (va.abs() @ v.abs().T)).cpu().numpy())
    mul, res, bias = _rows(2, (m, n), "bf16"), _rows(3, (m, n), "bf16"), _rows(4, (n,), "f32")
    acc, err = exact(vb)
    c, pre = mx.linear_fused("fprop", qa, qb, "bf16", bias=bias, activation="silu", mul=mul,
                             residual=res, save_pre=True)
    check_forward(c, pre, acc, err, "bf16", "silu", host64(bias), host64(mul), host64(res), "forward")
    acc, err = exact(vw)
    for u in (None, mul):
        got = mx.linear_act_backward(qa, qw, res, "gelu", mul=u, out_dtype="bf16")
        dz, dmul = got if u is not None else (got, None)
        check_backward(dz, dmul, acc, err, host64(res), "bf16", "gelu", host64(u), "backward")
    # the same by experts, whose columns begin inside the operand's tiles
    ends = torch.tensor([1000, 1003, 4200], dtype=torch.int32, device="cuda")
    w = new(3, n, k)
    qw = mx.quantize_grouped(w, dual=False)
    out = torch.full((m, n), 3.0, device="cuda")
    mx.linear_grouped("fprop", qa, qw.q1, ends, out=out)
    vw = torch.tensor(values(qw.q1), device="cuda").view(3, n, k)
    for e, (lo, hi) in enumerate(((0, 1000), (1000, 1003), (1003, 4200))):
        acc = (va[lo:hi] @ vw[e].T).cpu().numpy()
        err = (k / 128 + 10) * 2.0 ** -22 * (va[lo:hi].abs() @ vw[e].abs().T).cpu().numpy()
        check(out[lo:hi], acc, err, "f32", f"expert {e}")
    assert (out[4200:] == 3).all()


# ---- grouped ----------------------------------------------------------------

RAGGED = [300, 0, 5, 213, 130, 1, 500, 64]
GROUPS = [("fprop", RAGGED, 20, 2080, 160), ("dgrad", RAGGED, 20, 160, 2080),
          ("wgrad", RAGGED, 20, 768, 736), ("fprop", RAGGED, 20, 2112, 160),
          ("dgrad", RAGGED, 20, 160, 2112), ("wgrad", RAGGED, 20, 768, 768), ("fprop", [9] * 768, 3, 128, 64),
          ("fprop", [9] * 768, 3, 96, 64), ("wgrad", [9] * 50 + [0] * 718, 0, 64, 32),   # a full table
          ("fprop", [9] * 800, 0, 128, 64), ("dgrad", [9] * 800, 0, 64, 128),           # too many groups
          ("fprop", [2000, 3, 2300], 9, 2304, 32)]                                       # several tiles each


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("op,sizes,spare,out,cin", GROUPS)
def test_grouped(mx, op, sizes, spare, out, cin, dtype):
    import torch
    rng = np.random.Generator(np.random.PCG64(len(sizes) + out))
    t, e = sum(sizes) + spare, len(sizes)
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    rows = lambda c: mx.quantize_grouped(to_dev(activations_bf16(rng, (t, c), outlier_frac=0.01)),  # noqa: E731
                                         ends)
    if op == "wgrad":
        qa, qb = rows(out).q0, rows(cin).q0
    else:
        w = mx.quantize_grouped(to_dev(normal_bf16(rng, (e * out, cin), 0.05)).view(e, out, cin))
        qa, qb = (rows(cin).q1, w.q1) if op == "fprop" else (rows(out).q1, w.q0)
    shape = (e, out, cin) if op == "wgrad" else (t, out if op == "fprop" else cin)
    ref = _grouped_ref(op, qa, qb, oracle.group_ranges_ref(np.cumsum(sizes), t), out, cin)
    bias = _rows(21, (e, shape[-1]), "f32")
    mul, res = _rows(22, shape, dtype), _rows(23, shape, dtype)
    for b, act, u, r in ((None, "none", None, res), (bias, "silu", mul, None),
                         (bias, "gelu_tanh", mul, res)):
        c, pre = torch.full((2, *shape), 3.0, device="cuda").to(res.dtype)
        mx.linear_grouped(op, qa, qb, ends, out_dtype=dtype, bias=b, activation=act, mul=u,
                          residual=r, save_pre=pre, out=c)
        b64, u64, r64 = host64(b), host64(u), host64(r)
        for i, (at, acc, err) in enumerate(ref):
            pick = lambda v: None if v is None else v[at]  # noqa: E731
            check_forward(c[at], pre[at], acc, err, dtype, act, None if b is None else b64[i],
                          pick(u64), pick(r64), f"group {i}")
        if op != "wgrad":
            assert (c[sum(sizes):] == 3).all() and (pre[sum(sizes):] == 3).all()
    if op == "dgrad":
        pre, mul = _rows(32, shape, dtype), _rows(33, shape, dtype)
        for u in (None, mul):
            c, d = torch.full((2, *shape), 3.0, device="cuda").to(pre.dtype)
            mx.linear_act_backward(qa, qb, pre, "gelu", mul=u, ends=ends, out_dtype=dtype, out=c,
                                   dmul=None if u is None else d)
            p64, u64 = host64(pre), host64(u)
            for at, acc, err in ref:
                check_backward(c[at], d[at], acc, err, p64[at], dtype, "gelu",
                               None if u is None else u64[at], "backward")
            assert (c[sum(sizes):] == 3).all() and (d[sum(sizes):] == 3).all()


@pytest.mark.parametrize("out,cin", [(96, 64), (832, 736)])
def test_odd_widths(mx, out, cin):
    """Widths that no quantizer's blocks have along a row: the same operands,
    said to be narrower, give the same columns and write nothing beside them."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(out)
    sizes = [9, 0, 200, 40, 60, 70, 81]
    t, e = sum(sizes) + 5, len(sizes)
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    new = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    qx, qdy = mx.quantize_grouped(new(t, cin), ends), mx.quantize_grouped(new(t, out), ends)
    qw = mx.quantize_grouped(new(e, out, cin))

    def cut(q, rows, cols, **more):
        return mx.packed_operand(q.codes, q.scales, rows, cols, 0, groups=e, **more)
    o, c = out - 13, cin - 31
    want = mx.linear_grouped("wgrad", qdy.q0, qx.q0, ends)
    got = mx.linear_grouped("wgrad", cut(qdy.q0, t, o), cut(qx.q0, t, c), ends)
    assert torch.equal(got, want[:, :o, :c])
    want = mx.linear_grouped("dgrad", qdy.q1, qw.q0, ends)[:t - 5]
    wide = torch.full((t, cin), 5.0, device="cuda")
    mx.linear_grouped("dgrad", qdy.q1, cut(qw.q0, e * out, c, group_rows=out), ends, out=wide[:, :c])
    assert torch.equal(wide[:t - 5, :c], want[:, :c])
    assert (wide[:, c:] == 5).all() and (wide[t - 5:] == 5).all()


def test_nan_reaches_its_own_group_only(mx):
    import torch
    rng = np.random.Generator(np.random.PCG64(51))
    sizes, out, cin = [137, 240, 33, 90], 2560, 2048
    ends = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    x, dy = (to_dev(normal_bf16(rng, (520, c), 1.0)) for c in (cin, out))
    w = to_dev(normal_bf16(rng, (4 * out, cin), 1.0)).view(4, out, cin)
    x[138, 5], w[2, 7, 9], x[515] = float("nan"), float("inf"), float("nan")
    qx, qdy, qw = mx.quantize_grouped(x, ends), mx.quantize_grouped(dy, ends), mx.quantize_grouped(w)
    for op, a, b, shape, at in (("fprop", qx.q1, qw.q1, (500, out), [(138, slice(None)),
                                                                     (slice(377, 410), 7)]),
                                ("dgrad", qdy.q1, qw.q0, (500, cin), [(slice(377, 410), 9)]),
                                ("wgrad", qdy.q0, qx.q0, (4, out, cin), [(1, slice(None), 5)])):
        want = torch.zeros(shape, dtype=torch.bool, device="cuda")
        for i in at:
            want[i] = True
        got = mx.linear_grouped(op, a, b, ends).isnan()
        assert torch.equal(got if op == "wgrad" else got[:500], want), op


def test_captured_and_replayed(mx):
    """Graphs of grouped products with other ends and operands at each replay."""
    import torch
    t, out, cin = 1200, 2080, 128
    ends = torch.zeros(6, dtype=torch.int32, device="cuda")
    x = torch.zeros(t, cin, dtype=torch.bfloat16, device="cuda")
    w = mx.quantize_grouped(torch.randn(6, out, cin, device="cuda").bfloat16())
    outs = [[torch.zeros(t, out, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            for _ in range(3)]

    def step(c):
        q = mx.quantize_grouped(x, ends)
        mx.linear_grouped("fprop", q.q1, w.q1, ends, "bf16", activation="silu", save_pre=c[1], out=c[0])
        return mx.linear_grouped("wgrad", mx.quantize_grouped(c[0], ends).q0, q.q0, ends)
    step(outs[2])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dw = step(outs[i])
        graphs.append((g, dw))
    for split in ([1, 1, 400, 401, 900, 1200], [200, 400, 600, 800, 1000, 1100], [0, 0, 0, 0, 1200, 1200],
                  [0] * 6):
        ends.copy_(torch.tensor(split))
        x.normal_()
        for i, (g, dw) in enumerate(graphs):
            for c in outs[i] + outs[2]:
                c.zero_()
            g.replay()
            want = step(outs[2])
            torch.cuda.synchronize()
            assert torch.equal(dw, want), (split, i)
            assert all(torch.equal(a, b) for a, b in zip(outs[i], outs[2])), (split, i)


# ---- offsets past 31 and 32 bits ----------------------------------------------

@pytest.mark.parametrize("op,dtype", [("fprop", "bf16"), ("dgrad", "f32")])
def test_offsets_of_large_outputs(mx, op, dtype):
    """4.6 and 9.2 GB of output, in tiles: A's rows repeat every 256, so C's do."""
    import torch
    m, n, k = 70144, 32768, 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(256, k, generator=gen, device="cuda").bfloat16()
    w = torch.randn((n, k) if op == "fprop" else (k, n), generator=gen, device="cuda").bfloat16()
    qb = mx.quantize(w, 1 if op == "fprop" else 0)
    qa = mx.quantize(x.repeat(m // 256, 1), 1)
    acc, err = product(values(mx.quantize(x, 1)), values(qb))
    c = mx.linear_fused(op, qa, qb, out_dtype=dtype, activation="relu")
    check_forward(c[:256], None, acc, err, dtype, "relu", None, None, None, op)
    for i in range(0, m, 256 * 8):
        part = c[i:i + 256 * 8].view(-1, 256, n)
        assert (part == c[:256]).all(), i
    if op == "fprop":                            # a handful of rows a group: the few-rows kernel
        e = 11
        ends = torch.arange(1, e + 1, dtype=torch.int32, device="cuda") * 7
        big = torch.empty(1 << 32, dtype=torch.bfloat16, device="cuda").view(128, -1)
        out = big[:77, -n:]                      # rows 64 MB apart, 4.3 GB to the last
        qw = mx.packed_operand(qb.codes, qb.scales, n, k, 1, groups=1, group_rows=n)
        mx.linear_grouped("fprop", mx.quantize(x[:77], 1), qw, ends[-1:], out_dtype="bf16", out=out)
        check_forward(out, None, acc[:77], err[:77], "bf16", "none", None, None, None, "few rows")


def test_rows_far_apart(mx):
    """Rows of C, mul and the residual 17 MB apart (read and written by columns)."""
    import torch
    m, n, k = 1100, 3920, 96
    qa, qb, acc, err = _pair(mx, 4, "fprop", m, n, k)
    far = torch.empty(m * (1 << 23) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    views = [far.as_strided((m, n), (1 << 23, 1), 5000 * i) for i in range(3)]
    mul, res = _rows(2, (m, n), "bf16"), _rows(3, (m, n), "bf16")
    views[0].copy_(mul)
    views[1].copy_(res)
    mx.linear_fused("fprop", qa, qb, out_dtype="bf16", activation="silu", mul=views[0],
                    residual=views[1], out=views[2])
    check_forward(views[2], None, acc, err, "bf16", "silu", None, host64(mul), host64(res), "far")
    assert torch.equal(views[0], mul) and torch.equal(views[1], res)


def test_offsets_of_a_large_quantizer_source(mx):
    """3.9 GB of rows, through an index too: the ordinary quantizer's bytes."""
    import torch
    t, c = 60416, 32768
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(t, c, generator=gen, device="cuda", dtype=torch.bfloat16)
    ends = torch.tensor([t], dtype=torch.int32, device="cuda")
    want = [mx.quantize(x, a) for a in (1, 0)]
    for index in (None, torch.arange(t, device="cuda")):
        q = mx.quantize_grouped(x, ends, index=index)
        for got, ref in zip((q.q1, q.q0), want):
            assert torch.equal(got.codes, ref.codes) and torch.equal(got.scales, ref.scales)
