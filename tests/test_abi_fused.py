"""Host-side checks of the products with an epilogue, the grouped products and the
grouped quantizer: every invalid argument is refused before any HIP call. No GPU;
the addresses are never touched."""
import ctypes

import pytest
import torch

import mxfp4_microscaled_precision_amd as mx

P = 1 << 20         # fake, aligned addresses
F32, BF16 = 0, 1
GROUPED = mx.AXIS_GROUPED


@pytest.fixture(scope="module")
def lib():
    return mx.load_library()


def _q(rows, cols, axis, **f):
    q = mx.QTensorDesc(P, P, rows, cols, axis, 32, 1, 0, 0, 0)
    for k, v in f.items():
        setattr(q, k, v)
    return q


def _epilogue(**f):
    e = mx.EpilogueDesc(0, 0, None, 0, None, None, None, None, 256, 256, 256, 256)
    for k, v in f.items():
        setattr(e, k, v)
    return e


def _fused(lib, op=0, a=None, b=None, c=2 * P, ldc=256, dtype=BF16, e=None, **f):
    a = _q(64, 128, 1) if a is None else a
    b = _q(256, 128, 1) if b is None else b
    e = _epilogue(**f) if e is None else e
    return lib.mx_linear_fused(op, a, b, e, c, ldc, dtype, None)


EPILOGUES = [
    (-4, dict(activation=5)), (-4, dict(activation=-1)), (-4, dict(gradient=2)),
    (-4, dict(bias=P, bias_dtype=2)), (-3, dict(bias=P + 1, bias_dtype=BF16)),
    (-3, dict(bias=P + 2, bias_dtype=F32)),
    (-2, dict(mul=P, ldmul=255)), (-2, dict(residual=P, ldres=255)), (-2, dict(pre=P, ldpre=255)),
    (-3, dict(mul=P + 1)), (-3, dict(residual=P + 1)), (-3, dict(pre=P + 1)),
    (-4, dict(dmul=P)), (-4, dict(dmul=P, mul=3 * P)),                     # forward
    (-4, dict(pre=2 * P)),                                                # two outputs at one place
    (-2, dict(residual=2 * P, ldres=264)), (-2, dict(mul=2 * P, ldmul=264)),
    (-2, dict(pre=3 * P, mul=3 * P, ldmul=264)),
    (-1, dict(gradient=1)),                                               # no pre
    (-4, dict(gradient=1, pre=P, bias=P)), (-4, dict(gradient=1, pre=P, residual=P)),
    (-4, dict(gradient=1, pre=P, dmul=4 * P)),                            # no mul
    (-4, dict(gradient=1, pre=P, mul=3 * P, dmul=2 * P)),                 # C itself
    (-2, dict(gradient=1, pre=P, mul=3 * P, dmul=4 * P, lddmul=255)),
    (-2, dict(gradient=1, pre=2 * P, ldpre=264)),
    (-6, dict(mul=P, ldmul=1 << 60)),
]


@pytest.mark.parametrize("want,args", EPILOGUES)
def test_epilogue_refused(lib, want, args):
    assert _fused(lib, **args) == want
    ga = mx.GroupedDesc(_q(64, 128, 1), 4, -1)
    gb = mx.GroupedDesc(_q(1024, 128, 1), 4, 256)
    assert lib.mx_linear_grouped(0, ga, gb, P, _epilogue(**args), 2 * P, 256, BF16, None) == want


@pytest.mark.parametrize("want,args", [
    (-4, dict(op=3)), (-4, dict(dtype=2)), (-1, dict(c=None)), (-3, dict(c=2 * P + 1)),
    (-2, dict(ldc=255)), (-4, dict(op=1)),                                # axes of another op
    (-2, dict(b=_q(256, 160, 1))), (-5, dict(b=_q(256, 128, 1, rotate=3))),
    (-6, dict(a=_q(64, 128, 1, format=1), b=_q(256, 128, 1, format=1))),  # MXFP8
    (-4, dict(a=_q(64, 128, GROUPED))),
])
def test_fused_refused(lib, want, args):
    assert _fused(lib, **args) == want


def test_fused_null_operands(lib):
    assert lib.mx_linear_fused(0, None, _q(256, 128, 1), None, P, 256, BF16, None) == -1
    assert lib.mx_linear_fused(0, _q(64, 128, 1), None, None, P, 256, BF16, None) == -1


def test_empty_products_launch_nothing(lib):
    assert _fused(lib, a=_q(0, 128, 1), c=None) == 0
    assert _fused(lib, b=_q(0, 128, 1), c=None, ldc=0) == 0
    ga, gb = mx.GroupedDesc(_q(0, 128, 1), 4, -1), mx.GroupedDesc(_q(1024, 128, 1), 4, 256)
    assert lib.mx_linear_grouped(0, ga, gb, None, None, None, 256, BF16, None) == 0


def _grouped(lib, op=0, rows=64, groups=4, out=256, cin=128, ends=P, c=2 * P, ldc=None, dtype=BF16,
             a=None, b=None, **f):
    parts = {0: ((rows, cin, 1, -1), (groups * out, cin, 1, out)),
             1: ((rows, out, 1, -1), (groups * out, cin, GROUPED, out)),
             2: ((rows, out, GROUPED, -1), (rows, cin, GROUPED, -1))}[op]
    ga, gb = (mx.GroupedDesc(_q(r, k, axis), groups, each) for r, k, axis, each in parts)
    for g, fields in ((ga, a), (gb, b)):
        for k, v in (fields or {}).items():
            setattr(g.q if hasattr(g.q, k) else g, k, v)
    n = out if op == 0 else cin
    return lib.mx_linear_grouped(op, ga, gb, ends, _epilogue(**f), c, n if ldc is None else ldc,
                                 dtype, None)


@pytest.mark.parametrize("op", [0, 1, 2])
@pytest.mark.parametrize("want,args", [
    (-1, dict(ends=None)), (-3, dict(ends=P + 2)), (-1, dict(c=None)), (-3, dict(c=2 * P + 1)),
    (-4, dict(dtype=3)), (-2, dict(ldc=64)),
    (-4, dict(a=dict(axis=0))), (-4, dict(b=dict(axis=0))), (-4, dict(a=dict(block=16))),
    (-4, dict(a=dict(group_rows=16))),                     # rows are ragged
    (-4, dict(a=dict(groups=0))), (-4, dict(b=dict(group_rows=-2))),
    (-2, dict(a=dict(groups=5))), (-6, dict(a=dict(groups=65537))),
    (-5, dict(a=dict(rotate=0))), (-6, dict(a=dict(format=1))), (-4, dict(b=dict(rotate=9))),
    (-1, dict(a=dict(codes=None))), (-1, dict(b=dict(scales=None))),
    (-3, dict(a=dict(codes=P + 8))), (-3, dict(b=dict(scales=P + 2))),
    (-2, dict(a=dict(rows=-1))), (-2, dict(b=dict(cols=-32))),
])
def test_grouped_refused(lib, op, want, args):
    if args == dict(b=dict(group_rows=-2)) and op == 2:
        want = -4
    assert _grouped(lib, op, **args) == want


def test_grouped_extents_and_groups(lib):
    assert _grouped(lib, 0, a=dict(cols=160)) == -2
    assert _grouped(lib, 1, a=dict(cols=160)) == -2
    assert _grouped(lib, 2, b=dict(rows=65)) == -2
    assert _grouped(lib, 0, b=dict(group_rows=255)) == -2   # rows != groups * group_rows
    assert _grouped(lib, 0, b=dict(group_rows=-1)) == -4
    assert _grouped(lib, 2, b=dict(group_rows=16)) == -4
    # seeds matter for random signs only
    sign = dict(rotate=2)
    assert _grouped(lib, 2, a=dict(seed=1, **sign), b=dict(seed=2, **sign)) == -5


def test_operands_above_the_limit(lib):
    big = dict(rows=1 << 23, cols=256)
    assert _grouped(lib, 2, rows=1 << 23, out=256, cin=256) == -6
    assert mx.quantize_grouped_sizes(64, 128, 4)[0] == 256 * 128 * ((64 + 508) // 128) // 2
    assert big["rows"] * 256 // 2 >= 1 << 30


def test_sizes(lib):
    assert mx.quantize_grouped_sizes(300, 96, 3, -1, 1) == (512 * 128 // 2, 512 * 128 // 32)
    assert mx.quantize_grouped_sizes(300, 96, 3) == (256 * 128 * 5 // 2, 256 * 128 * 5 // 32)
    assert mx.quantize_grouped_sizes(600, 96, 3, 200) == (256 * 128 * 6 // 2, 256 * 128 * 6 // 32)
    assert mx.quantize_grouped_sizes(0, 96, 3) == (0, 0)
    assert mx.quantize_grouped_sizes(300, 83, 3) == mx.quantize_grouped_sizes(300, 96, 3)
    for args, want in [((64, 48, 4, -1, 1), -2), ((-1, 64, 4), -2), ((64, 64, 0), -4), ((64, 64, 4, -2), -4),
                       ((64, 64, 4, 15), -2), ((64, 64, 4, 16, 0), -4), ((64, 64, 65537), -6),
                       ((1 << 32, 64, 4), -6)]:
        with pytest.raises(mx.MxError) as ei:
            mx.quantize_grouped_sizes(*args)
        assert ei.value.status == want, args


def _quantize(lib, block=32, rot=1, rnd=0, c1=P, s1=P, c0=P, s0=P, sums=None, work=None, size=0,
              null=False, **f):
    s = mx.GroupedSourceDesc(P, 64, 96, 96, None, 0, 64, 4, -1, P)
    for k, v in f.items():
        setattr(s, k, v)
    return lib.mx_quantize_grouped(None if null else s, block, rot, rnd, 1, 2, c1, s1, c0, s0, sums,
                                   work, size, None, None, None)


NEED = 4 * 96 * 4       # four slices of 96 columns


@pytest.mark.parametrize("want,args", [
    (-1, dict(null=True)), (-4, dict(block=16)), (-4, dict(rot=4)), (-4, dict(rnd=2)),
    (-4, dict(groups=0)), (-4, dict(group_rows=-2)), (-2, dict(group_rows=15)),
    (-6, dict(groups=65537)), (-2, dict(rows=-1)), (-2, dict(cols=48)), (-2, dict(src_rows=-1)),
    (-2, dict(src_rows=63)),                               # without an index: the rows themselves
    (-4, dict(index=P, index_bits=16)), (-3, dict(index=P + 4, index_bits=64)),
    (-3, dict(index=P + 2, index_bits=32)),
    (-1, dict(x=None)), (-1, dict(c1=None)), (-1, dict(s1=None)), (-1, dict(c0=None)),
    (-1, dict(s0=None)), (-1, dict(ends=None)), (-3, dict(ends=P + 2)),
    (-2, dict(ld=95)), (-3, dict(ld=100)), (-3, dict(x=P + 8)), (-3, dict(c1=P + 8)),
    (-3, dict(s1=P + 2)), (-3, dict(c0=P + 8)), (-3, dict(s0=P + 1)),
    (-2, dict(sums=P, work=P, size=NEED - 1)), (-1, dict(sums=P, work=None, size=NEED)),
    (-3, dict(sums=P + 2, work=P, size=NEED)), (-3, dict(sums=P, work=P + 8, size=NEED)),
    (-6, dict(rows=1 << 24, src_rows=1 << 24, cols=128, ld=128)),
    (-6, dict(src_rows=1 << 33, index=P, index_bits=64)), (-6, dict(ld=1 << 60)),
])
def test_quantize_refused(lib, want, args):
    assert _quantize(lib, **args) == want


def test_quantize_empty_fills_descriptors(lib):
    s = mx.GroupedSourceDesc(None, 0, 64, 64, None, 0, 0, 3, -1, P)
    d1, d0 = mx.GroupedDesc(), mx.GroupedDesc()
    assert lib.mx_quantize_grouped(s, 32, 2, 1, 7, 8, None, None, P, P, None, None, 0, d1, d0,
                                   None) == 0
    assert (d1.q.rows, d1.q.cols, d1.q.axis, d1.q.rotate, d1.q.round, d1.q.seed) == (0, 64, 1, 2, 1, 7)
    assert (d0.q.axis, d0.q.seed, d0.groups, d0.group_rows) == (GROUPED, 8, 3, -1)


def test_grouped_operands_are_refused_elsewhere(lib):
    q = _q(64, 128, GROUPED)
    assert lib.mx_linear(2, q, q, P, 128, F32, None) == -4
    assert lib.mx_dequantize(q, P, 128, None) == -4


def test_binding_refuses_on_the_host():
    """The binding's own checks, on CPU tensors."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mx.quantize_grouped(x, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="bfloat16"):
        mx.quantize_grouped(x.float(), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        mx.packed_operand(torch.zeros(16384, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8),
                          64, 128, 1)


@pytest.mark.gpu
def test_binding_refuses(mx):
    def operand(rows, cols, axis=1):
        return mx.quantize(torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda"), axis)
    a, b = operand(4, 64), operand(32, 64)
    m = torch.zeros(4, 32, device="cuda")
    ends = torch.tensor([1, 4], dtype=torch.int32, device="cuda")
    w = mx.quantize_grouped(torch.zeros(2, 32, 64, dtype=torch.bfloat16, device="cuda"))
    rows = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: mx.linear_fused("fprop", a, b, mul=m[:, :31]),
        lambda: mx.linear_fused("fprop", a, b, mul=m.bfloat16()),
        lambda: mx.linear_fused("fprop", a, b, residual=m.cpu()),
        lambda: mx.linear_fused("fprop", a, b, residual=m.t().contiguous().t()),
        lambda: mx.linear_fused("fprop", a, b, bias=torch.zeros(31, device="cuda")),
        lambda: mx.linear_fused("fprop", a, b, bias=torch.zeros(64, device="cuda")[::2]),
        lambda: mx.linear_fused("fprop", a, b, bias=torch.zeros(32, device="cuda").half()),
        lambda: mx.linear_fused("fprop", a, b, out=m.bfloat16()),
        lambda: mx.linear_fused("fprop", a, w.q0),
        lambda: mx.linear_grouped("fprop", a, b, ends),
        lambda: mx.linear_grouped("fprop", a, w.q1, ends.long()),
        lambda: mx.linear_grouped("fprop", a, w.q1, ends[:1]),
        lambda: mx.linear_grouped("fprop", a, w.q1, ends.cpu()),
        lambda: mx.linear_grouped("fprop", a, w.q1, ends, bias=torch.zeros(32, device="cuda")),
        lambda: mx.quantize_grouped(rows),
        lambda: mx.quantize_grouped(rows, ends.long()),
        lambda: mx.quantize_grouped(rows, ends, index=torch.zeros(4, device="cuda")),
        lambda: mx.quantize_grouped(rows, ends, index=torch.zeros(4, 1, device="cuda").long()),
        lambda: mx.quantize_grouped(rows[None], ends),
        lambda: mx.quantize_grouped(torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")[:, :4]),
        lambda: mx.packed_operand(a.codes, a.scales[:3], 4, 64, 1),
        lambda: mx.packed_operand(a.codes, a.scales, 4, 64, 2, groups=2),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i}")
    with pytest.raises(KeyError):
        mx.linear_fused("fprop", a, b, activation="tanh")
    for call in (lambda: mx.linear_act_backward(a, operand(64, 32, 0), None, "silu"),
                 lambda: mx.linear_fused("fprop", a, b, out=m, save_pre=m)):
        with pytest.raises(mx.MxError):
            call()
