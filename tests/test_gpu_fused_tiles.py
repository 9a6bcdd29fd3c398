"""The kernel of 256x256 tiles, by calls that are held to it: columns that end
inside 64 and rows far apart (read and written element by element there), weight
and input gradients of experts of any width, a full table of groups, outputs
written over what they were computed from, repeated, replayed and concurrent
calls.

A narrow call's sums are those of the same operands said to be wider, added in
the same order, and its epilogue the same operations, so its outputs are the
wider call's columns bit for bit; the wider calls' accesses are whole units,
which other tests hold against fp64."""
import numpy as np
import pytest

import oracle
from datagen import activations_bf16, normal_bf16
from fused_util import check_backward, check_forward, host64, values
from gpu_util import to_dev
from launch_util import only_tiles
from test_gpu_fused import _grouped_ref, _rows

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16"]


def _tiles(call):
    """call(), which must be one launch of the tile kernel."""
    assert only_tiles(call), "another kernel"
    return call()


def _new(seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()


def _ends(sizes):
    import torch
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")


def _full(shape, dtype, value=7.0):
    import torch
    return torch.full(shape, value, device="cuda",
                      dtype=torch.float32 if dtype == "f32" else torch.bfloat16)


# ---- columns that end inside 64 ----------------------------------------------

M, N, WIDE, K = 4224, 4331, 4352, 4608      # 168 GFLOP


@pytest.mark.parametrize("dtype", DTYPES)
def test_columns_that_end_inside_64(mx, dtype):
    """Every epilogue with mul, residual and pre; rows at even and odd addresses."""
    import torch
    new = _new(1)
    qa, qb = mx.quantize(new(M, K), 1), mx.quantize(new(WIDE, K), 1)
    narrow = mx.packed_operand(qb.codes, qb.scales, N, K, 1)
    bias = _rows(2, (WIDE,), "f32")
    mul, res = _rows(3, (M, WIDE), dtype), _rows(4, (M, WIDE), dtype)
    for act, what in (("silu", "bmrp"), ("gelu", "mp"), ("relu", "rp"), ("gelu_tanh", "bm"),
                      ("none", "mr"), ("silu", "")):
        b, u, r = (x if c in what else None for c, x in zip("bmr", (bias, mul, res)))
        pre = "p" in what
        want = _tiles(lambda: mx.linear_fused("fprop", qa, qb, dtype, bias=b, activation=act, mul=u,
                                              residual=r, save_pre=pre))
        out = _full((2, M, WIDE), dtype)
        cut = lambda t: None if t is None else t[..., :N].contiguous() if t.dim() == 1 else t[:, :N]  # noqa: E731
        got = _tiles(lambda: mx.linear_fused("fprop", qa, narrow, dtype, bias=cut(b), activation=act,
                                             mul=cut(u), residual=cut(r), out=out[0][:, :N],
                                             save_pre=out[1][:, :N] if pre else False))
        for g, w, o in zip(got if pre else (got,), want if pre else (want,), out):
            assert torch.equal(g, w[:, :N]), f"{act} {what}"
            assert (o[:, N:] == 7).all(), f"{act} {what}: beside the matrix"


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_columns_that_end_inside_64(mx, dtype):
    import torch
    new = _new(5)
    qa, qb = mx.quantize(new(M, K), 1), mx.quantize(new(K, WIDE), 0)
    narrow = mx.packed_operand(qb.codes, qb.scales, K, N, 0)
    pre, mul = _rows(6, (M, WIDE), dtype), _rows(7, (M, WIDE), dtype)
    for act, u in (("silu", mul), ("gelu", None), ("gelu_tanh", mul), ("relu", mul), ("none", None)):
        want = _tiles(lambda: mx.linear_act_backward(qa, qb, pre, act, mul=u, out_dtype=dtype))
        out = _full((2, M, WIDE), dtype)
        got = _tiles(lambda: mx.linear_act_backward(
            qa, narrow, pre[:, :N], act, mul=None if u is None else u[:, :N], out_dtype=dtype,
            out=out[0][:, :N], dmul=None if u is None else out[1][:, :N]))
        for g, w, o in zip((got,) if u is None else got, (want,) if u is None else want, out):
            assert torch.equal(g, w[:, :N]), act
            assert (o[:, N:] == 7).all(), act


def test_columns_that_end_inside_64_in_fp64(mx):
    """fp32 with both matrices and its gradient with dmul."""
    import torch
    new = _new(8)
    qa, qb, qw = mx.quantize(new(M, K), 1), mx.quantize(new(N, K), 1), mx.quantize(new(K, N), 0)
    va, vb, vw = (torch.tensor(values(q), device="cuda") for q in (qa, qb, qw))

    def exact(v):
        return ((va @ v.T).cpu().numpy(),
                ((K / 128 + 10) * 2.0 ** -22 * (va.abs() @ v.abs().T)).cpu().numpy())
    bias, mul, res = _rows(9, (N,), "f32"), _rows(10, (M, N), "f32"), _rows(11, (M, N), "f32")
    acc, err = exact(vb)
    c, pre = _tiles(lambda: mx.linear_fused("fprop", qa, qb, bias=bias, activation="gelu_tanh", mul=mul,
                                            residual=res, save_pre=True))
    check_forward(c, pre, acc, err, "f32", "gelu_tanh", host64(bias), host64(mul), host64(res), "forward")
    acc, err = exact(vw)
    dz, dmul = _tiles(lambda: mx.linear_act_backward(qa, qw, res, "silu", mul=mul))
    check_backward(dz, dmul, acc, err, host64(res), "f32", "silu", host64(mul), "backward")


def _cut(mx, q, rows, cols, axis=0, **more):
    return mx.packed_operand(q.codes, q.scales, rows, cols, axis, **more)


@pytest.mark.parametrize("dtype", DTYPES)
def test_weight_gradients_of_any_width(mx, dtype):
    """164 GFLOP; three experts, one without rows, whose matrices end inside a
    tile both ways; onto the output itself."""
    import torch
    new = _new(12)
    sizes, spare, out, cin = [3001, 0, 5899], 100, 2112, WIDE
    t, ends = sum(sizes) + spare, _ends(sizes)
    qa, qb = mx.quantize_grouped(new(t, out), ends).q0, mx.quantize_grouped(new(t, cin), ends).q0
    o, c = out - 13, N
    na, nb = _cut(mx, qa, t, o, groups=3), _cut(mx, qb, t, c, groups=3)
    mul, res = _rows(13, (3, out, cin), dtype), _rows(14, (3, out, cin), dtype)
    inner = lambda x: x[:, :o, :c].contiguous()  # noqa: E731
    for u, act in ((None, "none"), (mul, "silu")):
        want = _tiles(lambda: mx.linear_grouped("wgrad", qa, qb, ends, dtype, activation=act, mul=u,
                                                residual=res))
        got, m = inner(res), None if u is None else inner(u)
        _tiles(lambda: mx.linear_grouped("wgrad", na, nb, ends, dtype, activation=act, mul=m,
                                         residual=got, out=got))
        assert torch.equal(got, inner(want)), act
        assert torch.equal(got[1], inner(res)[1]) or act != "none"
    # columns of a wider buffer: nothing beside them is written
    buf = _full((3, o, cin + 3), dtype)
    _tiles(lambda: mx.linear_grouped("wgrad", na, nb, ends, dtype, out=buf[:, :, 1:c + 1]))
    want = mx.linear_grouped("wgrad", qa, qb, ends, dtype)
    assert torch.equal(buf[:, :, 1:c + 1], want[:, :o, :c])
    assert (buf[:, :, 0] == 7).all() and (buf[:, :, c + 1:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_input_gradients_of_any_width(mx, dtype):
    """167 GFLOP; experts whose rows begin inside a tile, rows of no expert."""
    import torch
    new = _new(15)
    sizes, spare, out = [1000, 3, 3677], 20, 4096
    t, ends, live = sum(sizes) + spare, _ends(sizes), sum(sizes)
    qa = mx.quantize(new(t, out), 1)
    qb = mx.quantize_grouped(new(3, out, WIDE)).q0
    narrow = _cut(mx, qb, 3 * out, N, groups=3, group_rows=out)
    mul, res = _rows(16, (t, WIDE), dtype), _rows(17, (t, WIDE), dtype)

    def compare(call, pairs):
        want = _tiles(lambda: call(qb, WIDE, None, None))
        o = _full((2, t, WIDE), dtype)
        got = _tiles(lambda: call(narrow, N, o[0][:, :N], o[1][:, :N] if pairs else None))
        for g, w, b in zip(got if pairs else (got,), want if pairs else (want,), o):
            assert torch.equal(g[:live], w[:live, :N])
            assert (b[live:] == 7).all() and (b[:, N:] == 7).all()
    for u, r in ((None, res), (mul, res), (mul, None)):
        compare(lambda b, n, c, second: mx.linear_grouped(
            "dgrad", qa, b, ends, dtype, activation="gelu", mul=None if u is None else u[:, :n],
            residual=None if r is None else r[:, :n], out=c,
            save_pre=True if second is None else second), True)
        compare(lambda b, n, c, second: mx.linear_act_backward(
            qa, b, res[:, :n], "silu", mul=None if u is None else u[:, :n], ends=ends,
            out_dtype=dtype, out=c, dmul=second), u is not None)


def test_experts_whose_columns_begin_anywhere(mx):
    """Forward with bias, mul, residual and pre: expert e's columns begin at row
    4331 e of the operand, inside a tile's 64."""
    import torch
    new = _new(18)
    sizes, k = [1000, 3, 3197], K
    t, ends = sum(sizes) + 24, _ends(sizes)
    qa = mx.quantize(new(t, k), 1)
    qw = mx.quantize_grouped(new(3, N, k), dual=False).q1
    bias, mul, res = _rows(19, (3, N), "f32"), _rows(20, (t, N), "bf16"), _rows(21, (t, N), "bf16")
    out = _full((2, t, N), "bf16")
    _tiles(lambda: mx.linear_grouped("fprop", qa, qw, ends, "bf16", bias=bias, activation="silu",
                                     mul=mul, residual=res, save_pre=out[1], out=out[0]))
    va = torch.tensor(values(qa), device="cuda")
    vw = torch.tensor(values(qw), device="cuda").view(3, N, k)
    b64, u64, r64 = host64(bias), host64(mul), host64(res)
    for e, (lo, hi) in enumerate(oracle.group_ranges_ref(ends.tolist(), t)):
        acc = (va[lo:hi] @ vw[e].T).cpu().numpy()
        err = (k / 128 + 10) * 2.0 ** -22 * (va[lo:hi].abs() @ vw[e].abs().T).cpu().numpy()
        check_forward(out[0, lo:hi], out[1, lo:hi], acc, err, "bf16", "silu", b64[e], u64[lo:hi],
                      r64[lo:hi], f"expert {e}")
    assert (out[:, sum(sizes):] == 7).all()


# ---- rows 16 MB apart: no 32-bit offsets, so element by element ----------------

def _far(dtype, rows, n, count):
    """`count` matrices of `rows` rows of n, 16 MB from row to row, in one buffer
    of sevens, each beginning at an odd element."""
    ld = 1 << (22 if dtype == "f32" else 23)
    buf = _full((rows, ld), dtype)
    return buf, [buf[:, 1 + i * (n + 65):][:, :n] for i in range(count)]


def _gaps(buf, n, count):
    """What lies before, between and behind those matrices is untouched."""
    edges = [0] + [1 + i * (n + 65) + n for i in range(count)]
    return all((buf[:, e:e + (65 if i else 1)] == 7).all() for i, e in enumerate(edges))


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_far_apart(mx, dtype):
    import torch
    m, n, k = 300, 16384, 16416             # 162 GFLOP
    new = _new(22)
    qa, qb = mx.quantize(new(m, k), 1), mx.quantize(new(n, k), 1)
    bias, mul, res = _rows(23, (n,), "f32"), _rows(24, (m, n), dtype), _rows(25, (m, n), dtype)
    buf, (u, r, c, pre) = _far(dtype, m, n, 4)
    u.copy_(mul)
    r.copy_(res)
    want = _tiles(lambda: mx.linear_fused("fprop", qa, qb, dtype, bias=bias, activation="gelu", mul=mul,
                                          residual=res, save_pre=True))
    _tiles(lambda: mx.linear_fused("fprop", qa, qb, dtype, bias=bias, activation="gelu", mul=u,
                                   residual=r, save_pre=pre, out=c))
    assert torch.equal(c, want[0]) and torch.equal(pre, want[1])
    assert torch.equal(u, mul) and torch.equal(r, res) and _gaps(buf, n, 4)
    # the gradient: pre is read from r, dz and dmul written over the others
    qb = mx.quantize(new(k, n), 0)
    want = _tiles(lambda: mx.linear_act_backward(qa, qb, res, "silu", mul=mul, out_dtype=dtype))
    _tiles(lambda: mx.linear_act_backward(qa, qb, r, "silu", mul=u, out_dtype=dtype, out=c, dmul=pre))
    assert torch.equal(c, want[0]) and torch.equal(pre, want[1])
    assert torch.equal(u, mul) and torch.equal(r, res) and _gaps(buf, n, 4)


def test_rows_far_apart_of_experts(mx):
    """Forward over ragged rows and weight gradients, matrix after matrix."""
    import torch
    n, k = 16384, 16416
    new = _new(26)
    ends, m = _ends([140, 150]), 300
    qa, qb = mx.quantize(new(m, k), 1), mx.quantize_grouped(new(2, n, k), dual=False).q1
    mul = _rows(27, (m, n), "bf16")
    buf, (u, c) = _far("bf16", m, n, 2)
    u.copy_(mul)
    want = _tiles(lambda: mx.linear_grouped("fprop", qa, qb, ends, "bf16", activation="silu", mul=mul))
    _tiles(lambda: mx.linear_grouped("fprop", qa, qb, ends, "bf16", activation="silu", mul=u, out=c))
    assert torch.equal(c[:290], want[:290]) and (c[290:] == 7).all() and _gaps(buf, n, 2)
    del qa, qb, want
    t, out = 33000, 150
    ends = _ends([20001, 12990])
    qa = mx.quantize_grouped(new(t, 160), ends).q0
    qa, qb = _cut(mx, qa, t, out, groups=2), mx.quantize_grouped(new(t, n), ends).q0
    buf.fill_(7)
    three = lambda v: v.as_strided((2, out, n), (out * v.stride(0), v.stride(0), 1))  # noqa: E731
    u.copy_(mul)
    want = _tiles(lambda: mx.linear_grouped("wgrad", qa, qb, ends, "bf16", mul=mul.view(2, out, n)))
    _tiles(lambda: mx.linear_grouped("wgrad", qa, qb, ends, "bf16", mul=three(u), out=three(c)))
    assert torch.equal(c, want.view(m, n)) and torch.equal(u, mul) and _gaps(buf, n, 2)


# ---- in place, special values, the table ---------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [4352, 4331])
def test_gradient_written_over_what_it_reads(mx, n, dtype):
    """dz over pre and dmul over mul, in whole units and by columns."""
    import torch
    new = _new(28)
    qa, qb = mx.quantize(new(M, K), 1), mx.quantize(new(K, n), 0)
    pre, mul = _rows(29, (M, n), dtype), _rows(30, (M, n), dtype)
    for act in ("silu", "gelu"):
        want = _tiles(lambda: mx.linear_act_backward(qa, qb, pre, act, mul=mul, out_dtype=dtype))
        p, u = pre.clone(), mul.clone()
        _tiles(lambda: mx.linear_act_backward(qa, qb, p, act, mul=u, out_dtype=dtype, out=p, dmul=u))
        assert torch.equal(p, want[0]) and torch.equal(u, want[1]), act
        p, u = pre.clone(), mul.clone()         # the other way round
        _tiles(lambda: mx.linear_act_backward(qa, qb, p, act, mul=u, out_dtype=dtype, out=u, dmul=p))
        assert torch.equal(u, want[0]) and torch.equal(p, want[1]), act


@pytest.mark.parametrize("dtype", DTYPES)
def test_grouped_outputs_written_over_what_they_read(mx, dtype):
    """Groups that begin inside a tile's 64 rows."""
    import torch
    new = _new(31)
    sizes, t, out, cin = [301, 1, 0, 515, 77, 300], 1300, 2112, 2304
    ends, live = _ends(sizes), sum(sizes)
    w = mx.quantize_grouped(new(6, out, cin))
    qdy, qx = mx.quantize(new(t, out), 1), mx.quantize(new(t, cin), 1)
    pre, mul = _rows(32, (t, cin), dtype), _rows(33, (t, cin), dtype)
    want = _full((2, t, cin), dtype)
    _tiles(lambda: mx.linear_act_backward(qdy, w.q0, pre, "silu", mul=mul, ends=ends, out_dtype=dtype,
                                          out=want[0], dmul=want[1]))
    p, u = pre.clone(), mul.clone()
    _tiles(lambda: mx.linear_act_backward(qdy, w.q0, p, "silu", mul=u, ends=ends, out_dtype=dtype,
                                          out=p, dmul=u))
    for got, ref, before in ((p, want[0], pre), (u, want[1], mul)):
        assert torch.equal(got[:live], ref[:live]) and torch.equal(got[live:], before[live:])
    # forward: C over mul, pre over the residual
    mul, res = _rows(34, (t, out), dtype), _rows(35, (t, out), dtype)
    want = _full((2, t, out), dtype)
    _tiles(lambda: mx.linear_grouped("fprop", qx, w.q1, ends, dtype, activation="gelu", mul=mul,
                                     residual=res, save_pre=want[1], out=want[0]))
    u, r = mul.clone(), res.clone()
    _tiles(lambda: mx.linear_grouped("fprop", qx, w.q1, ends, dtype, activation="gelu", mul=u,
                                     residual=r, save_pre=r, out=u))
    for got, ref, before in ((u, want[0], mul), (r, want[1], res)):
        assert torch.equal(got[:live], ref[:live]) and torch.equal(got[live:], before[live:])


def test_nan_reaches_its_own_group_only(mx):
    import torch
    rng = np.random.Generator(np.random.PCG64(51))
    sizes, t, out, cin = [437, 640, 133, 290], 1520, 2560, 2048
    ends = _ends(sizes)
    x, dy = (to_dev(normal_bf16(rng, (t, c), 1.0)) for c in (cin, out))
    w = to_dev(normal_bf16(rng, (4 * out, cin), 1.0)).view(4, out, cin)
    x[438, 5], w[2, 7, 9], x[1515] = float("nan"), float("inf"), float("nan")
    qx, qdy, qw = mx.quantize_grouped(x, ends), mx.quantize_grouped(dy, ends), mx.quantize_grouped(w)
    own = slice(1077, 1210)
    for op, a, b, shape, at in (("fprop", qx.q1, qw.q1, (1500, out), [(438, slice(None)), (own, 7)]),
                                ("dgrad", qdy.q1, qw.q0, (1500, cin), [(own, 9)]),
                                ("wgrad", qdy.q0, qx.q0, (4, out, cin), [(1, slice(None), 5)])):
        want = torch.zeros(shape, dtype=torch.bool, device="cuda")
        for i in at:
            want[i] = True
        got = _tiles(lambda: mx.linear_grouped(op, a, b, ends)).isnan()
        assert torch.equal(got if op == "wgrad" else got[:1500], want), op


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("groups", [768, 769])
def test_weight_gradients_of_a_full_table(mx, groups, dtype):
    """768 groups fill the table of the tile kernel's groups; one more is the
    other kernel's."""
    import torch
    rng = np.random.Generator(np.random.PCG64(groups))
    out, cin = 128, 64
    sizes = [(0, 9, 1, 130, 17)[i % 5] for i in range(groups)]
    t, ends = sum(sizes) + 3, _ends(sizes)
    qa, qb = (mx.quantize_grouped(to_dev(activations_bf16(rng, (t, c), outlier_frac=0.01)), ends).q0
              for c in (out, cin))
    ref = _grouped_ref("wgrad", qa, qb, oracle.group_ranges_ref(ends.tolist(), t), out, cin)
    mul, res = _rows(36, (groups, out, cin), dtype), _rows(37, (groups, out, cin), dtype)
    call = lambda: mx.linear_grouped("wgrad", qa, qb, ends, dtype, activation="gelu_tanh",  # noqa: E731
                                     mul=mul, residual=res, save_pre=True)
    assert only_tiles(call) == (groups == 768)
    c, pre = call()
    acc, err = (np.stack([r[i] for r in ref]) for i in (1, 2))
    check_forward(c, pre, acc, err, dtype, "gelu_tanh", None, host64(mul), host64(res), "table")
    assert all(torch.equal(g, p) for _ in range(10) for g, p in zip(call(), (c, pre)))


# ---- repeated, replayed, side by side ------------------------------------------

E, T, D, F = 6, 1500, 2304, 2112
SPLITS = ([1, 1, 400, 401, 900, 1500], [200, 400, 600, 800, 1000, 1100], [0, 0, 0, 0, 1500, 1500],
          [0] * 6, [301, 302, 302, 817, 894, 1480])


def _layer_weights(mx):
    new = _new(38)
    return mx.quantize_grouped((0.1 * new(E, F, D)))


def _layer(mx, w, x, u, ends, out, products=None):
    """Gate, its gradient and the weight gradient; the outputs. `products` is
    given each product to call."""
    call = products or (lambda f: f())
    qx = mx.quantize_grouped(x, ends)
    h, pre = call(lambda: mx.linear_grouped("fprop", qx.q1, w.q1, ends, "bf16", activation="silu",
                                            mul=u, save_pre=out[1], out=out[0]))
    qh = mx.quantize_grouped(h, ends)
    dx = call(lambda: mx.linear_grouped("dgrad", qh.q1, w.q0, ends, "f32", residual=out[2], out=out[2]))
    dz, du = call(lambda: mx.linear_act_backward(qh.q1, w.q0, x, "gelu", mul=x, ends=ends,
                                                 out_dtype="bf16", out=out[3], dmul=out[4]))
    dw = call(lambda: mx.linear_grouped("wgrad", qh.q0, qx.q0, ends, out_dtype="bf16"))
    return [h, pre, dx, dz, du, dw]


def _layer_buffers():
    import torch
    return ([torch.zeros(T, F, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            + [torch.zeros(T, D, device="cuda")]
            + [torch.zeros(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)])


def _layer_inputs(seed, split):
    import torch
    new = _new(seed)
    return new(T, D), new(T, F), torch.tensor(split, dtype=torch.int32, device="cuda")


def test_the_layer_s_products_are_tiles(mx):
    x, u, ends = _layer_inputs(39, SPLITS[0])
    _layer(mx, _layer_weights(mx), x, u, ends, _layer_buffers(), _tiles)


@pytest.mark.parametrize("split", SPLITS)
def test_same_bits_every_time(mx, split):
    import torch
    w = _layer_weights(mx)
    x, u, ends = _layer_inputs(40, split)
    want = _layer(mx, w, x, u, ends, _layer_buffers())
    for i in range(10):
        got = _layer(mx, w, x, u, ends, _layer_buffers())
        for j, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), f"run {i}, output {j}"


def test_captured_and_replayed(mx):
    """Two graphs, replayed in turn with other rows and ends, eager work between."""
    import torch
    w, graphs = _layer_weights(mx), []
    for seed in (41, 42):
        x, u, ends = _layer_inputs(seed, SPLITS[0])
        out = _layer_buffers()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            got = _layer(mx, w, x, u, ends, out)
        graphs.append((g, x, u, ends, out, got))
    for step, split in enumerate(SPLITS * 2):
        for k, (g, x, u, ends, out, got) in enumerate(graphs):
            for t, v in zip((x, u, ends), _layer_inputs(50 + 2 * step + k, split)):
                t.copy_(v)
            for o in out:
                o.zero_()
            g.replay()
            want = _layer(mx, w, x, u, ends, _layer_buffers())
            torch.cuda.synchronize()
            for j, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), f"step {step}, graph {k}, output {j}"


@pytest.mark.parametrize("raw", [False, True])
def test_side_by_side(mx, raw):
    """The same products on two streams at once, each with its own ends."""
    import torch
    w = _layer_weights(mx)
    cases = [_layer_inputs(60 + i, SPLITS[(0, 4)[i]]) for i in range(2)]
    qs = [mx.quantize_grouped(x, ends) for x, _, ends in cases]

    outs = [[(torch.zeros_like(u), torch.zeros_like(u)) for _ in range(11)] for _, u, _ in cases]

    def gate(i, n, stream=None):
        _, u, ends = cases[i]
        c, pre = outs[i][n]
        return mx.linear_grouped("fprop", qs[i].q1, w.q1, ends, "bf16", activation="silu", mul=u,
                                 save_pre=pre, out=c, stream=stream)
    want = [_tiles(lambda i=i: gate(i, 10)) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for n in range(10):
        for i, s in enumerate(streams):
            gate(i, n, s.cuda_stream if raw else s)
    torch.cuda.synchronize()
    for i in range(2):
        for n, (c, pre) in enumerate(outs[i]):
            assert torch.equal(c, want[i][0]) and torch.equal(pre, want[i][1]), (i, n)


# ---- nothing to sum ------------------------------------------------------------

@pytest.mark.parametrize("m,n,tiles", [(5, 40, False), (1100, 3136, True)])
def test_no_reduction(mx, m, n, tiles):
    """K == 0, by experts: the sums are zeros, the epilogue's terms remain."""
    import torch
    ends = _ends([m // 2, m - m // 2 - 2])
    a = mx.quantize(torch.empty((m, 0), dtype=torch.bfloat16, device="cuda"), 1)
    w = mx.quantize_grouped(torch.empty((2, n, 0), dtype=torch.bfloat16, device="cuda")).q1
    bias, res = _rows(70, (2, n), "f32"), _rows(71, (m, n), "f32")
    out = _full((m, n), "f32")
    call = lambda: mx.linear_grouped("fprop", a, w, ends, bias=bias, activation="relu",  # noqa: E731
                                     residual=res, out=out)
    assert only_tiles(call) == tiles
    call()
    for e, (lo, hi) in enumerate(((0, m // 2), (m // 2, m - 2))):
        assert torch.equal(out[lo:hi], bias[e].clamp(min=0) + res[lo:hi])
    assert (out[m - 2:] == 7).all()


@pytest.mark.parametrize("out,cin,tiles", [(33, 32, False), (2112, 2304, True)])
@pytest.mark.parametrize("rows", [0, 5])
def test_weight_gradients_of_no_rows(mx, rows, out, cin, tiles):
    """No row at all, or none that is an expert's: the residual."""
    import torch
    ends = _ends([0, 0])
    new = _new(72)
    qa, qb = (mx.quantize_grouped(new(rows, c), ends).q0 for c in (-(-out // 32) * 32, cin))
    qa = _cut(mx, qa, rows, out, groups=2)
    res = _rows(73, (2, out, cin), "f32")
    call = lambda: mx.linear_grouped("wgrad", qa, qb, ends, residual=res)  # noqa: E731
    assert only_tiles(call) == tiles
    assert torch.equal(call(), res)
