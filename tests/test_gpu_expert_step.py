"""The grouped operators together, as a training step of a layer of experts runs
them: rows gathered in the router's order, gate and up projections, the gated
activation, the down projection; backward through all of it, weight gradients
summed over two micro-batches. Every call is checked against fp64 fed with that
call's own inputs (the GPU's outputs of the step before). Then the same calls in
captured graphs, on other streams and side by side."""
import numpy as np
import pytest

import oracle
from fused_util import check, check_backward, check_forward, host64, product, values
from gpu_util import host_u8

pytestmark = pytest.mark.gpu

E, D, F, TOKENS = 5, 96, 160, 150


def _weights(mx, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: (0.1 * torch.randn(s, generator=gen, device="cuda")).bfloat16()  # noqa: E731
    return [mx.quantize_grouped(w) for w in (new(E, F, D), new(E, F, D), new(E, D, F))]


def _route(seed):
    """Two experts a token: the rows' tokens by expert, and the experts' ends."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    score = torch.randn(TOKENS, E, generator=gen, device="cuda")
    score[:, 3] = -100                                  # an expert nobody wants
    pick = score.topk(2, 1).indices.flatten()
    order = pick.argsort(stable=True)
    ends = torch.bincount(pick, minlength=E).cumsum(0).to(torch.int32)
    return order // 2, ends


def _groups(a, b, op, ends, n):
    """[(place, acc, bound)] of a grouped product of the packed operands."""
    at, found, va, vb = 0, [], values(a), values(b)
    each = b.group_rows
    kp = -(-each // 128) * 128 if each > 0 else 0
    for e, (lo, hi) in enumerate(oracle.group_ranges_ref(ends.tolist(), n)):
        deep = -(-(hi - lo) // 128) * 128
        if op == "fprop":
            found.append((slice(lo, hi), *product(va[lo:hi], vb[e * each:(e + 1) * each])))
        elif op == "dgrad":
            found.append((slice(lo, hi), *product(va[lo:hi], vb[:, e * kp:e * kp + va.shape[1]])))
        else:
            found.append((e, *product(va[:, at:at + deep], vb[:, at:at + deep])))
        at += deep
    return found


def test_training_step(mx):
    import torch
    wg, wu, wd = _weights(mx, 1)
    grads = [torch.zeros(s, device="cuda") for s in ((E, F, D), (E, F, D), (E, D, F))]
    n = 2 * TOKENS
    for batch in range(2):
        index, ends = _route(batch)
        gen = torch.Generator(device="cuda").manual_seed(10 + batch)
        x = torch.randn(TOKENS, D, generator=gen, device="cuda").bfloat16()
        dy = (1e-2 * torch.randn(n, D, generator=gen, device="cuda")).bfloat16()
        # forward
        qx = mx.quantize_grouped(x, ends, index=index)
        u = mx.linear_grouped("fprop", qx.q1, wu.q1, ends, "bf16")
        h, pre = mx.linear_grouped("fprop", qx.q1, wg.q1, ends, "bf16", activation="silu", mul=u,
                                   save_pre=True)
        qh = mx.quantize_grouped(h, ends)
        y = mx.linear_grouped("fprop", qh.q1, wd.q1, ends, "bf16")
        for at, acc, err in _groups(qx.q1, wu.q1, "fprop", ends, n):
            check(u[at], acc, err, "bf16", "up")
        for at, acc, err in _groups(qx.q1, wg.q1, "fprop", ends, n):
            check_forward(h[at], pre[at], acc, err, "bf16", "silu", None, host64(u)[at], None, "gate")
        for at, acc, err in _groups(qh.q1, wd.q1, "fprop", ends, n):
            check(y[at], acc, err, "bf16", "down")
        # backward
        qdy = mx.quantize_grouped(dy, ends, sums=True)
        dz, du = mx.linear_act_backward(qdy.q1, wd.q0, pre, "silu", mul=u, ends=ends,
                                        out_dtype="bf16")
        for at, acc, err in _groups(qdy.q1, wd.q0, "dgrad", ends, n):
            check_backward(dz[at], du[at], acc, err, host64(pre)[at], "bf16", "silu",
                           host64(u)[at], "gate")
        qdz, qdu = mx.quantize_grouped(dz, ends), mx.quantize_grouped(du, ends)
        part = mx.linear_grouped("dgrad", qdz.q1, wg.q0, ends, "f32")
        dx = mx.linear_grouped("dgrad", qdu.q1, wu.q0, ends, "f32", residual=part)
        for at, acc, err in _groups(qdu.q1, wu.q0, "dgrad", ends, n):
            check_forward(dx[at], None, acc, err, "f32", "none", None, None, host64(part)[at], "dx")
        for grad, a, b in zip(grads, (qdz, qdu, qdy), (qx, qx, qh)):
            before = host64(grad)
            mx.linear_grouped("wgrad", a.q0, b.q0, ends, residual=grad, out=grad)
            for e, acc, err in _groups(a.q0, b.q0, "wgrad", ends, n):
                check_forward(grad[e], None, acc, err, "f32", "none", None, None, before[e], "dw")
        assert not grads[0][3].any()                    # the idle expert


def _layer(mx, w, x, index, ends, out):
    """Forward and backward of one layer; a list of all its outputs."""
    qx = mx.quantize_grouped(x, ends, index=index, sums=True)
    h, pre = mx.linear_grouped("fprop", qx.q1, w[0].q1, ends, "bf16", activation="gelu",
                               save_pre=True, out=out[0])
    qh = mx.quantize_grouped(h, ends)
    y = mx.linear_grouped("fprop", qh.q1, w[2].q1, ends, "bf16", out=out[1])
    qy = mx.quantize_grouped(y, ends, sums=True)
    dz = mx.linear_act_backward(qy.q1, w[2].q0, pre, "gelu", ends=ends, out_dtype="bf16", out=out[2])
    dw = mx.linear_grouped("wgrad", qy.q0, qh.q0, ends)
    return [qx.sums, h, y, qy.sums, dz, dw, qx.q0.codes, qx.q0.scales]


def _buffers(n):
    import torch
    return [torch.zeros(n, c, dtype=torch.bfloat16, device="cuda") for c in (F, D, F)]


def test_captured_and_replayed(mx):
    """Two graphs, replayed in turn with other rows and ends, eager work between."""
    import torch
    w, n = _weights(mx, 2), 2 * TOKENS
    graphs = []
    for seed in (3, 4):
        index, ends = _route(seed)
        x = torch.zeros(TOKENS, D, dtype=torch.bfloat16, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _layer(mx, w, x, index, ends, _buffers(n))
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        out = _buffers(n)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = _layer(mx, w, x, index, ends, out)
        graphs.append((g, x, index, ends, out, got))
    for step in range(4):
        for k, (g, x, index, ends, out, got) in enumerate(graphs):
            i, e = _route(20 + 2 * step + k)
            index.copy_(i)
            ends.copy_(e if step < 3 else e.clamp(max=200))      # rows of no expert
            x.normal_()
            for o in out:
                o.zero_()
            g.replay()
            want = _layer(mx, w, x, index, ends, _buffers(n))
            torch.cuda.synchronize()
            for j, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a, b), f"step {step}, graph {k}, output {j}"


@pytest.mark.parametrize("raw", [False, True])
def test_on_other_streams(mx, raw):
    """Two layers at once on streams of their own give what one after the other
    gives, bit for bit."""
    import torch
    w, n = _weights(mx, 5), 2 * TOKENS
    cases = []
    for seed in (6, 7):
        index, ends = _route(seed)
        cases.append((torch.randn(TOKENS, D, device="cuda").bfloat16(), index, ends))
    want = [_layer(mx, w, *c, _buffers(n)) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    keep = []
    for _ in range(3):
        for s, (x, index, ends) in zip(streams, cases):
            h = s.cuda_stream if raw else s
            qx = mx.quantize_grouped(x, ends, index=index, sums=True, stream=h)
            y = torch.zeros(n, F, dtype=torch.bfloat16, device="cuda")
            torch.cuda.current_stream().synchronize()    # y is ready there
            mx.linear_grouped("fprop", qx.q1, w[0].q1, ends, "bf16", activation="gelu", out=y,
                              stream=h)
            keep.append((qx, y))
    torch.cuda.synchronize()
    for i, (qx, y) in enumerate(keep):
        assert torch.equal(qx.sums, want[i % 2][0]) and torch.equal(y, want[i % 2][1])


def test_same_bits_every_time(mx):
    """Large enough for many workgroups: no order of theirs shows."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(8)
    t, e = 3000, 7
    x = torch.randn(t, 512, generator=gen, device="cuda").bfloat16()
    w = torch.randn(e, 768, 512, generator=gen, device="cuda").bfloat16()
    ends = torch.tensor([100, 100, 900, 1500, 1501, 2600, 2990], dtype=torch.int32, device="cuda")
    qw = mx.quantize_grouped(w)
    runs = []
    for _ in range(3):
        q = mx.quantize_grouped(x, ends, sums=True)
        y = torch.zeros(t, 768, device="cuda")
        mx.linear_grouped("fprop", q.q1, qw.q1, ends, activation="silu", out=y)
        runs.append((q.sums, y, mx.linear_grouped("wgrad", q.q0, q.q0, ends)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_operands_from_existing_buffers(mx):
    """Operands made again from their buffers, as after a checkpoint."""
    import torch
    w, n = _weights(mx, 9), 2 * TOKENS
    index, ends = _route(9)
    x = torch.randn(n, D, device="cuda").bfloat16()
    q = mx.quantize_grouped(x, ends)

    def again(t, axis):
        return mx.packed_operand(t.codes.clone(), t.scales.clone(), *t.source_shape, axis,
                                 groups=t.groups, group_rows=t.group_rows)
    y = torch.zeros(2, n, F, device="cuda")
    mx.linear_grouped("fprop", q.q1, w[0].q1, ends, out=y[0])
    mx.linear_grouped("fprop", again(q.q1, 1), again(w[0].q1, 1), ends, out=y[1])
    assert torch.equal(y[0], y[1])
    a = mx.linear_grouped("wgrad", q.q0, q.q0, ends)
    b = mx.linear_grouped("wgrad", again(q.q0, 0), again(q.q0, 0), ends)
    assert torch.equal(a, b)
    one = mx.quantize(x, 1)
    assert torch.equal(mx.linear("fprop", one, mx.quantize(x, 1)),
                       mx.linear("fprop", mx.packed_operand(one.codes, one.scales, n, D, 1), one))
    assert np.array_equal(host_u8(one.codes), host_u8(q.q1.codes))
