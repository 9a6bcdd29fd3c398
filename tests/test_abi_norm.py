"""Host-side checks of the norm, its gradient and clipping: every invalid
argument is refused before any HIP call, and a set's table is laid out as the
kernels read it. No GPU; the addresses are never touched."""
import ctypes

import numpy as np
import pytest
import torch  # noqa: F401  (the library must bind to torch's HIP runtime)

import mxfp4_microscaled_precision_amd as mx

P = 4096            # a fake, aligned address
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    return mx.load_library()


def _norm(lib, fmt=1, block=32, rot=1, rnd=0, c1=P, s1=P, c0=None, s0=None, d1=None, d0=None,
          null=False, **f):
    n = mx.NormDesc(P, P, P, P, P, 64, 64, 64, 64, 64, BF16, F32, 1e-5)
    for k, v in f.items():
        setattr(n, k, v)
    return lib.mx_rmsnorm_quantize(None if null else ctypes.byref(n), fmt, block, rot, rnd, 5, 6,
                                   c1, s1, c0, s0, d1, d0, None)


@pytest.mark.parametrize("want,args", [
    (-1, dict(null=True)),
    (-4, dict(block=16)), (-4, dict(rot=4)), (-4, dict(rnd=2)), (-4, dict(fmt=2)),
    (-4, dict(fmt=1, rnd=1)),                                   # E4M3 rounds to nearest only
    (-4, dict(dtype=2)), (-4, dict(weight_dtype=-1)),
    (-4, dict(eps=-1e-9)), (-4, dict(eps=float("nan"))), (-4, dict(eps=float("inf"))),
    (-2, dict(rows=-1)), (-2, dict(cols=48)), (-2, dict(rows=48, c0=P, s0=P)),
    (-2, dict(ldx=32)), (-2, dict(ldr=32)), (-2, dict(ldh=32)),
    (-2, dict(ldr=128)),                                        # h is the residual: same pitch
    (-3, dict(ldx=68)), (-3, dict(dtype=F32, ldx=66)), (-3, dict(x=P + 8)), (-3, dict(h=P + 2)),
    (-3, dict(residual=P + 4)), (-3, dict(weight=P + 8)), (-3, dict(rstd=P + 2)),
    (-3, dict(c1=P + 8)), (-3, dict(s1=P + 2)), (-3, dict(c0=P + 8, s0=P)),
    (-3, dict(c0=P, s0=P + 1)),
    (-1, dict(x=None)), (-1, dict(h=None)), (-1, dict(weight=None)), (-1, dict(rstd=None)),
    (-1, dict(c1=None)), (-1, dict(s1=None)), (-1, dict(c0=P)), (-1, dict(s0=P)),
    (-6, dict(rows=1 << 17, cols=1 << 14, ldx=1 << 14, ldr=1 << 14, ldh=1 << 14, fmt=0)),
    (-6, dict(rows=1 << 16, cols=1 << 14, ldx=1 << 14, ldr=1 << 14, ldh=1 << 14)),
    (-6, dict(rows=(1 << 31) + 32)), (-6, dict(cols=1 << 36, ldx=1 << 36)),
    (-6, dict(rows=1 << 20, ldx=1 << 60)),
])
def test_rmsnorm_quantize_refuses(lib, want, args):
    assert _norm(lib, **args) == want


def test_rmsnorm_quantize_empty_fills_descriptors(lib):
    d1, d0 = mx.QTensorDesc(), mx.QTensorDesc()
    assert _norm(lib, rows=0, rot=3, c0=P, s0=P, d1=ctypes.byref(d1), d0=ctypes.byref(d0)) == 0
    assert (d1.rows, d1.cols, d1.axis, d1.rotate, d1.seed, d1.format) == (0, 64, 1, 3, 5, 1)
    assert (d0.rows, d0.cols, d0.axis, d0.rotate, d0.seed, d0.format) == (0, 64, 0, 3, 6, 1)
    assert _norm(lib, rows=3, cols=0, x=None, weight=None, c1=None, s1=None) == 0


def _back(lib, work=P, size=1 << 30, null=False, **f):
    g = mx.NormGradDesc(P, 2 * P, P, P, P, P, P, 64, 64, 64, 64, 64, 64, BF16, F32)
    for k, v in f.items():
        setattr(g, k, v)
    return lib.mx_rmsnorm_backward(None if null else ctypes.byref(g), work, size, None)


@pytest.mark.parametrize("want,args", [
    (-1, dict(null=True)), (-4, dict(dtype=3)), (-4, dict(weight_dtype=2)),
    (-4, dict(h=P)),                                            # dh over h
    (-2, dict(rows=-1)), (-2, dict(cols=60)), (-2, dict(lddy=32)), (-2, dict(ldh=32)),
    (-2, dict(ldres=32)), (-2, dict(lddh=32)), (-2, dict(lddh=128)), (-2, dict(rows=4096, size=4095)),
    (-1, dict(dy=None)), (-1, dict(h=None)), (-1, dict(rstd=None)), (-1, dict(weight=None)),
    (-1, dict(dh=None)), (-1, dict(dweight=None)), (-1, dict(rows=4096, work=None)),
    (-3, dict(dy=P + 8)), (-3, dict(h=P + 8)), (-3, dict(dres=P + 8)), (-3, dict(dh=P + 8)),
    (-3, dict(rstd=P + 2)), (-3, dict(weight=P + 8)), (-3, dict(dweight=P + 4)),
    (-3, dict(rows=4096, work=P + 8)), (-3, dict(lddy=68)), (-3, dict(dtype=F32, ldh=66)),
    (-6, dict(rows=(1 << 31) + 1)), (-6, dict(rows=1 << 20, ldh=1 << 60)),
])
def test_rmsnorm_backward_refuses(lib, want, args):
    assert _back(lib, **args) == want


def test_backward_workspace(lib):
    n = ctypes.c_size_t()
    assert lib.mx_rmsnorm_backward_workspace(7, 64, ctypes.byref(n)) == 0
    assert n.value == 0                                 # few rows: one launch, no partial rows
    assert lib.mx_rmsnorm_backward_workspace(700, 64, ctypes.byref(n)) == 0
    assert 700 * 64 * 4 >= n.value > 0 and n.value % (64 * 4) == 0
    assert lib.mx_rmsnorm_backward_workspace(1 << 30, 64, ctypes.byref(n)) == 0
    assert n.value <= 4096 * 64 * 4                     # bounded, whatever the rows
    assert lib.mx_rmsnorm_backward_workspace(7, 64, None) == -1
    assert lib.mx_rmsnorm_backward_workspace(-1, 64, ctypes.byref(n)) == -2
    assert lib.mx_rmsnorm_backward_workspace(1 << 40, 64, ctypes.byref(n)) == -6
    assert _back(lib, cols=0) == 0


def _fill(lib, entries, size=None):
    """(status, set, table, grads) of entries (data, rows, cols, ld, dtype)."""
    g = (mx.GradDesc * max(1, len(entries)))(*[mx.GradDesc(*e) for e in entries])
    need = ctypes.c_size_t()
    st = lib.mx_grad_set_size(len(entries), g, ctypes.byref(need))
    s = mx.GradSetDesc()
    if st != 0:
        return st, s, None, g
    host = np.zeros(max(1, need.value // 8 + 1), np.uint64)
    st = lib.mx_grad_set_fill(len(entries), g, host.ctypes.data,
                              need.value if size is None else size, ctypes.byref(s))
    return st, s, host, g


@pytest.mark.parametrize("want,entries", [
    (-4, [(P, 2, 8, 8, 2)]), (-2, [(P, -1, 8, 8, 0)]), (-2, [(P, 2, 8, 7, 0)]),
    (-1, [(None, 2, 8, 8, 0)]), (-3, [(P + 2, 2, 8, 8, 0)]), (-3, [(P + 1, 2, 8, 8, 1)]),
    (-6, [(P, 1 << 30, 8, 1 << 40, 0)]), (-6, [(P, 1 << 30, 1 << 31, 1 << 31, 0)]),
    (-4, [(P, 2, 8, 8, 0), (P + 32, 2, 8, 8, 0)]),              # overlap
    (-4, [(P, 2, 8, 8, 0), (P, 2, 8, 8, 0)]),                   # twice
    (-4, [(P, 2, 8, 16, 0), (P, 2, 8, 16, 0)]),                 # twice, with gaps
    (0, [(P, 2, 8, 8, 0), (P + 64, 2, 8, 8, 0)]),               # side by side
    (0, [(P, 2, 8, 16, 0), (P + 32, 2, 8, 16, 0)]),             # column slices of one buffer
    (0, [(None, 0, 8, 8, 0), (P + 2, 2, 8, 8, 1)]), (0, []),
])
def test_grad_set_checks(lib, want, entries):
    st, s, host, _ = _fill(lib, entries)
    assert st == want
    if want == 0:
        assert s.count == len(entries) and s.table is None


def test_grad_set_table(lib):
    """Tensors (address, rows, cols, ld, fp32), then (tensor, chunk) pairs that
    cover every element once, then the gapless tensors by address."""
    entries = [(P + 65536, 300, 100, 100, 0), (P, 3, 5, 9, 1), (None, 0, 4, 4, 0),
               (P + 4096, 1, 4097, 4097, 1)]
    st, s, host, _ = _fill(lib, entries)
    assert st == 0
    t = host[:20].reshape(4, 5).astype(np.int64)
    assert t[0].tolist() == [P + 65536, 300, 100, 100, 1]
    assert t[1].tolist() == [P, 3, 5, 9, 0]
    assert t[3].tolist() == [P + 4096, 1, 4097, 4097, 0]
    pairs = host[20:20 + s.chunks].view(np.uint32).reshape(-1, 2).tolist()
    want = [[i, j] for i, e in enumerate(entries) for j in range(-(-e[1] * e[2] // s.chunk))]
    assert pairs == want
    order = host[20 + s.chunks:].view(np.uint32)[:2].tolist()
    assert order == [3, 0]
    st, s, _, _ = _fill(lib, entries, size=8)
    assert st == -2


def _with_table(s, at=P):
    s.table = at
    return s


def test_grad_norm_and_clip_refuse(lib):
    W = lib.mx_grad_workspace()
    ok = [(P, 2, 8, 8, 0), (P + 64, 2, 8, 8, 1)]
    st, s, keep, g = _fill(lib, ok)
    ref = ctypes.byref
    assert lib.mx_grad_norm(ref(s), P, P, W, None) == -1        # table not uploaded
    _with_table(s)
    assert lib.mx_grad_norm(None, P, P, W, None) == -1
    assert lib.mx_grad_norm(ref(s), None, P, W, None) == -1
    assert lib.mx_grad_norm(ref(s), P, None, W, None) == -1
    assert lib.mx_grad_norm(ref(s), P, P, W - 1, None) == -2
    assert lib.mx_grad_norm(ref(s), P + 2, P, W, None) == -3
    assert lib.mx_grad_norm(ref(s), P, P + 4, W, None) == -3
    _with_table(s, P + 4)
    assert lib.mx_grad_norm(ref(s), P, P, W, None) == -3
    _with_table(s)
    for bad in (-1.0, float("nan")):
        assert lib.mx_grad_clip(ref(s), None, bad, P, P, W, None) == -4
    assert lib.mx_grad_clip(ref(s), None, 1.0, None, P, W, None) == -1
    bare = mx.GradSetDesc()
    bare.count = 3                                              # tensors, but no array of them
    assert lib.mx_grad_norm(ref(bare), P, P, W, None) == -1
    assert lib.mx_grad_clip(ref(s), ref(bare), 1.0, P, P, W, None) == -1
    far = P + (1 << 20)
    for want, other in [
            (-5, [(far, 2, 8, 8, 0)]), (-5, [(far, 2, 8, 8, 0), (far + 64, 2, 8, 8, 0)]),
            (-5, [(far, 4, 4, 4, 0), (far + 64, 2, 8, 8, 1)]),
            (-4, [(P + 32, 2, 8, 8, 0), (far, 2, 8, 8, 1)]),    # out[0] over in[0] and in[1]
            (-4, [(far, 2, 8, 8, 0), (P, 2, 8, 8, 1)])]:        # out[1] over in[0]
        st, o, k2, g2 = _fill(lib, other)
        assert st == 0
        assert lib.mx_grad_clip(ref(s), ref(_with_table(o)), 1.0, P, P, W, None) == want
    st, o, k2, g2 = _fill(lib, [(far, 2, 8, 8, 0), (far + 64, 2, 8, 8, 1)])
    assert lib.mx_grad_clip(ref(s), ref(o), 1.0, P, P, W, None) == -1   # out's table missing


def test_binding_refuses_before_the_library():
    """Shapes, types and devices the binding refuses by itself."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        mx.rmsnorm_quantize(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        mx.rmsnorm_backward(x, x, torch.ones(4), w)
    with pytest.raises(ValueError, match="CUDA"):
        mx.GradSet([w])
    with pytest.raises(ValueError, match="CUDA"):
        mx.clip_grad_norm([w], 1.0)
