"""Global gradient norm and clipping on the GPU against the oracle in fp64.

The norm's squares and sums are fp64, so it is one rounding to fp32 from the
oracle's: 2^-24, times 1.001 for the sum's own error (below 1e-9 here). coef
rounds once (2^-24), and so does its product with an element, to the tensor's
type: 2^-24 (fp32) or 2^-8 (bf16) of the result, or half the smallest
subnormal.
"""
import numpy as np
import pytest

import oracle
from norm_util import dev, host, values

pytestmark = pytest.mark.gpu


def _close(got, ref, bf16):
    step, tiny = (2.0 ** -8, 2.0 ** -134) if bf16 else (2.0 ** -24, 2.0 ** -150)
    bound = (step + 2.0 ** -24) * 1.001 * np.abs(ref) + tiny
    err = np.abs(host(got).astype(np.float64) - ref)
    assert np.all(err <= bound), f"{(err / bound).max():.3g} of the bound"


def _norm_close(got, ref):
    assert got.shape == () and abs(float(got) - ref) <= 1.001 * 2.0 ** -24 * ref


def _tensors(shapes, seed=0, scale=1e-3):
    """[(fp32 values, bf16?)] in alternating types."""
    rng = np.random.default_rng(seed)
    return [(values(rng, s, i % 2 == 1, scale), i % 2 == 1) for i, s in enumerate(shapes)]


SETS = [
    [(1,)], [(7,)], [(8,), (8,)], [(3, 5), (1, 1), (129,)],
    [(64, 64), (64,), (64, 64), (1000, 33), (33,)],
    [(2048,), (2049,), (2047, 1), (1, 2050)],
    [(517, 517), (129, 517), (1811, 517), (517,)] * 5,
    [(4, 3, 2), (2, 2, 2, 2), (0, 5), (0,), (6,)],
    [(3000, 1000), (900, 4096)],
]


@pytest.mark.parametrize("case", range(len(SETS)))
@pytest.mark.parametrize("limit", [0.25, 4.0])
def test_against_oracle(mx, case, limit):
    """limit: max_norm as a multiple of the norm."""
    ts = _tensors(SETS[case], case)
    vals = [v for v, _ in ts]
    norm = oracle.grad_norm_ref(vals)
    max_norm = float(np.float32(limit * norm))
    _, ref = oracle.clip_ref(vals, max_norm)
    grads = [dev(v, b) for v, b in ts]
    _norm_close(mx.grad_norm(grads), norm)
    out = [g.clone().fill_(9.0) for g in grads]
    _norm_close(mx.clip_grad_norm(grads, max_norm, out=out), norm)
    for o, g, r, (v, b) in zip(out, grads, ref, ts):
        assert np.array_equal(host(g), v)                 # the input stays
        _close(o, r, b)
    s = mx.GradSet(grads)
    _norm_close(mx.clip_grad_norm(s, max_norm), norm)
    for o, g, (v, b) in zip(out, grads, ts):
        assert np.array_equal(host(g), host(o))           # in place: the same bits
        if limit > 1:
            assert np.array_equal(host(g), v)
    if limit < 1:
        second = float(mx.grad_norm(s))
        # every element within 2^-8 + 2^-24 of its scaled value
        assert abs(second - limit * norm) <= (2.0 ** -8 + 2.0 ** -22) * limit * norm + 2e-6 * limit


def _flat(ts, align, bf16):
    """Views of one flat buffer, one after the other; the rest stays 3."""
    import torch
    at, n = [], 1
    for v in ts:
        n = -(-n // align) * align
        at.append(n)
        n += v.size
    flat = torch.full((n + 5,), 3.0, dtype=torch.bfloat16 if bf16 else torch.float32,
                      device="cuda")
    views = [flat[a:a + v.size].view(v.shape) for a, v in zip(at, ts)]
    for t, v in zip(views, ts):
        t.copy_(dev(v, bf16))
    keep = torch.ones_like(flat, dtype=torch.bool)
    for a, v in zip(at, ts):
        keep[a:a + v.size] = False
    return flat, views, keep


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("align_in,align_out", [(1, 1), (1, 8), (8, 1), (3, 1)])
def test_packed_without_alignment(mx, bf16, align_in, align_out):
    """Tensors at any element of a flat buffer; what lies between them and
    behind the last stays as it was."""
    import torch
    rng = np.random.default_rng(20)
    ts = [values(rng, s, bf16, 1e-2) for s in ((31, 67), (5,), (1,), (129, 255), (4097,), (2,))]
    flat, views, keep = _flat(ts, align_in, bf16)
    oflat, outs, okeep = _flat([0 * v for v in ts], align_out, bf16)
    norm, ref = oracle.clip_ref(ts, 0.5)
    _norm_close(mx.clip_grad_norm(views, 0.5, out=outs), norm)
    for o, r in zip(outs, ref):
        _close(o, r, bf16)
    mx.clip_grad_norm(views, 0.5)
    for o, g in zip(outs, views):
        assert torch.equal(o, g)
    assert torch.all(flat[keep] == 3.0) and torch.all(oflat[okeep] == 3.0)


def test_strided(mx):
    """Row-strided matrices (slices of wider buffers, a column, a strided
    vector) on either side; the gaps are neither read nor written."""
    import torch
    rng = np.random.default_rng(21)
    for bf16 in (True, False):
        shapes = [(130, 70), (3, 4099), (700, 1), (257, 9), (1, 50)]
        ts = [values(rng, s, bf16, 1e-2) for s in shapes]
        norm, ref = oracle.clip_ref(ts, 0.5)
        wide = [dev(v, bf16, v.shape[1] + 3) for v in ts]
        bigs = [torch.full((v.shape[0], v.shape[1] + 6), 5.0, dtype=wide[0].dtype, device="cuda")
                for v in ts]
        outs = [b[:, 2:2 + v.shape[1]] for b, v in zip(bigs, ts)]
        plain = [dev(v, bf16) for v in ts]
        flat_out = [torch.zeros_like(p) for p in plain]
        for src, dst in ((wide, outs), (plain, outs), (wide, flat_out)):
            for o in dst:
                o.fill_(1.0)
            _norm_close(mx.clip_grad_norm(src, 0.5, out=dst), norm)
            for o, r in zip(dst, ref):
                _close(o, r, bf16)
        mx.clip_grad_norm(wide, 0.5)
        for g, o in zip(wide, flat_out):
            assert torch.equal(g, o)
        for o in outs:
            o.fill_(5.0)
        assert all(torch.all(b == 5.0) for b in bigs)
    v = values(rng, (600,), False, 1e-2)
    base = torch.full((600, 3), float("nan"), device="cuda")
    base[:, 1] = torch.from_numpy(v).cuda()
    _norm_close(mx.grad_norm([base[:, 1]]), oracle.grad_norm_ref([v]))


def test_extreme_magnitudes(mx):
    """Squares beyond fp32's range on either side; subnormal elements."""
    import torch
    for scale in (1e30, 1e-30, 1e-41):
        v = (np.random.default_rng(22).standard_normal(5000) * scale).astype(np.float32)
        norm, ref = oracle.clip_ref([v], 1.0)
        g = torch.from_numpy(v.copy()).cuda()
        got = mx.clip_grad_norm([g], 1.0)
        assert abs(float(got) - norm) <= 1.001 * 2.0 ** -24 * norm + 2.0 ** -150
        _close(g, ref[0], False)
    big = torch.full((1 << 20,), 3e38, device="cuda")          # the norm itself overflows
    assert torch.isinf(mx.grad_norm([big]))


@pytest.mark.parametrize("bf16", [True, False])
def test_offsets_beyond_32_bits(mx, bf16):
    """A tensor of more than 4 GiB, without gaps and with: only a few elements,
    the first and last among them, are not zero."""
    import torch
    n = (1 << 32) // (2 if bf16 else 4) + 4099
    at = torch.tensor([0, 1, n // 2, n - 4100, n - 2, n - 1], device="cuda")
    v = torch.tensor([3.0, -4.0, 12.0, 1.0, 2.0, -2.0], device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    g[at] = v.to(g.dtype)
    norm = float(np.sqrt(178.0))
    _norm_close(mx.clip_grad_norm([g], 1.0), norm)
    _close(g[at], (v.double().cpu().numpy()) / (norm + 1e-6), bf16)
    assert int(torch.count_nonzero(g)) == 6
    g[at] = v.to(g.dtype)
    wide = g[:n // 64 * 64].view(-1, 64)[:, :33]            # the column slice's elements only
    keep = (at % 64 < 33) & (at < n // 64 * 64)
    norm = float(v[keep].double().square().sum().sqrt())
    _norm_close(mx.grad_norm([wide]), norm)


def test_nonfinite_and_limits(mx):
    import torch
    for bad in (float("nan"), float("inf"), float("-inf")):
        v = np.ones((3, 40), np.float32)
        v[1, 7] = bad
        w = np.full(9, 2.0, np.float32)
        norm, ref = oracle.clip_ref([v, w], 1.0)
        g = [dev(v, False), dev(w, True)]
        got = mx.clip_grad_norm(g, 1.0)
        assert np.array_equal(np.float32(float(got)), np.float32(norm), equal_nan=True)
        for a, r in zip(g, ref):
            assert np.array_equal(host(a), r.astype(np.float32), equal_nan=True)
    g = [dev(np.ones(100), False)]
    mx.clip_grad_norm(g, 0.0)
    assert not g[0].any()
    g = [dev(np.ones(100), False)]
    assert float(mx.clip_grad_norm(g, float("inf"))) == 10.0 and torch.all(g[0] == 1.0)
    z = [torch.zeros(50, device="cuda")]
    assert float(mx.clip_grad_norm(z, 1.0)) == 0.0 and not z[0].any()
    assert float(mx.grad_norm([])) == 0.0
    assert float(mx.clip_grad_norm([torch.empty(0, device="cuda")], 1.0)) == 0.0


def test_deterministic(mx):
    import torch
    ts = [dev(v, b) for v, b in _tensors([(1000, 517), (333, 4096), (77,)] * 3, 23)]
    s = mx.GradSet(ts)
    a, b = mx.grad_norm(s), mx.grad_norm(s)
    assert torch.equal(a, b)
    out1, out2 = ([torch.empty_like(t) for t in ts] for _ in range(2))
    mx.clip_grad_norm(s, 0.1, out=out1)
    mx.clip_grad_norm(s, 0.1, out=out2)
    assert all(torch.equal(x, y) for x, y in zip(out1, out2))


def test_streams_and_graphs(mx):
    """A set used on a side stream and in two captured graphs replayed in turn
    with eager calls between."""
    import torch
    ts = _tensors([(200, 300), (77,), (1000, 65)], 24)
    grads = [dev(v, b) for v, b in ts]
    outs = [[torch.zeros_like(g) for g in grads] for _ in range(3)]
    s, os = mx.GradSet(grads), [mx.GradSet(o) for o in outs]
    limits = (0.05, 0.2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = mx.clip_grad_norm(s, limits[0], out=os[0], stream=side)
    torch.cuda.synchronize()
    norm, ref = oracle.clip_ref([v for v, _ in ts], limits[0])
    _norm_close(n, norm)
    for o, r, (v, b) in zip(outs[0], ref, ts):
        _close(o, r, b)
    n = mx.clip_grad_norm(grads, limits[0], out=outs[1], stream=side.cuda_stream)   # lists
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[1]))
    graphs, norms = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(mx.clip_grad_norm(s, limits[i], out=os[i]))
        graphs.append(g)
    for k in range(3):
        for t, (v, b) in zip(grads, ts):
            t.copy_(dev(v * np.float32(2 ** k), b))
        for i in range(2):
            graphs[i].replay()
            n = mx.clip_grad_norm(s, limits[i], out=os[2])
            torch.cuda.synchronize()
            assert torch.equal(n, norms[i])
            assert all(torch.equal(a, b) for a, b in zip(outs[i], outs[2]))


def test_binding_refusals(mx):
    import torch
    a, b = torch.ones(4, 6, device="cuda"), torch.ones(6, 4, device="cuda")
    with pytest.raises(ValueError):
        mx.GradSet([a.half()])
    with pytest.raises(ValueError):
        mx.GradSet([a.t()])
    with pytest.raises(ValueError):
        mx.GradSet([torch.ones(2, 3, 4, device="cuda")[:, :, ::2]])
    for status, bad in ((-5, lambda: mx.clip_grad_norm([a], 1.0, out=[b])),
                        (-5, lambda: mx.clip_grad_norm([a], 1.0, out=[a.bfloat16()])),
                        (-4, lambda: mx.clip_grad_norm([a, a], 1.0)),
                        (-4, lambda: mx.clip_grad_norm([a[:2], a[2:]], 1.0, out=[a[2:], a[:2]])),
                        (-2, lambda: mx.grad_norm([a[:1].expand(4, 6)])),
                        (-4, lambda: mx.clip_grad_norm([a], -1.0))):
        with pytest.raises(mx.MxError) as e:
            bad()
        assert e.value.status == status
    assert torch.all(a == 1.0)
    # the same tensors in another set: in place, tensor by tensor
    mx.clip_grad_norm(mx.GradSet([a]), 1.0, out=mx.GradSet([a]))
    assert abs(float(mx.grad_norm([a])) - 1.0) < 1e-5


@pytest.mark.parametrize("bf16", [True, False])
def test_no_limit(mx, bf16):
    """An infinite max_norm scales nothing, also where the norm is infinite; a
    NaN norm still shows in every element."""
    import torch
    v = np.ones((3, 40), np.float32)
    v[1, 7], v[2, 3] = np.inf, -np.inf
    norm, ref = oracle.clip_ref([v], float("inf"))
    assert np.isinf(norm) and np.array_equal(ref[0], v)
    g, out = [dev(v, bf16)], [dev(0 * np.ones_like(v), bf16)]
    assert torch.isinf(mx.clip_grad_norm(g, float("inf"), out=out))
    assert np.array_equal(host(out[0]), v)
    assert torch.isinf(mx.clip_grad_norm(g, float("inf")))
    assert np.array_equal(host(g[0]), v)
    v[0, 0] = np.nan
    g = [dev(v, bf16)]
    assert torch.isnan(mx.clip_grad_norm(g, float("inf"))) and torch.isnan(g[0]).all()
    assert np.isnan(oracle.clip_ref([v], float("inf"))[1][0]).all()
