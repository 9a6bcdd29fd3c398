"""Cases and plain forms of the products with an epilogue, of the products
grouped by expert, and of the grouped quantizer.

A feed-forward layer, dense or of experts, is products whose outputs go through
a bias, an activation, a gate and a residual sum. Four operators cover that:

  fused     C = act(A B^T + bias) * mul + residual over two packed MXFP4
            operands; A B^T + bias is kept where a backward pass follows.
  back      the gradient through the activation in the epilogue of the input
            gradient's product: g = A B^T, C = g * mul * act'(pre) and
            dmul = g * act(pre).
  experts   the same products with one matrix per expert: rows [ends[e - 1],
            ends[e]) of A meet expert e's matrix (fprop, dgrad), or their sum
            over those rows is expert e's weight gradient (wgrad).
  quantize  rows gathered in the router's order and quantized in both
            orientations, where the blocks along the rows never cross from one
            expert to the next; and the column sums of each expert's rows (the
            gradient of its bias).

`run` computes them from elementary torch operations; with `own` set it calls
the package's entry points. Operand buffers are in their packed tile order;
those that `quantize` writes are compared as the values they hold: E2M1 codes
as float8 values (which hold every E2M1 value), scales as float8_e8m0fnu.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# the axis of each operand that its blocks run along
AXES = {"fprop": (1, 1), "dgrad": (1, 0), "wgrad": (0, 0)}


def _fused(name, kind, m, n, k, **more):
    """C [m, n] with reduction extent k."""
    return {"name": name, "op": "fused", "kind": kind, "m": m, "n": n, "k": k, "dtype": "bf16",
            "bias": False, "act": "none", "mul": False, "residual": False, "pre": False, **more}


def _back(name, m, n, k, **more):
    return {"name": name, "op": "back", "kind": "dgrad", "m": m, "n": n, "k": k, "dtype": "bf16",
            "act": "silu", "mul": False, **more}


def _experts(name, kind, experts, rows, n, k, **more):
    """fprop, dgrad: C [rows, n], reduction extent k; wgrad: C [experts, n, k],
    summed over an expert's rows."""
    return {"name": name, "op": "experts", "kind": kind, "experts": experts, "rows": rows, "n": n,
            "k": k, "dtype": "bf16", "bias": False, "act": "none", "mul": False,
            "residual": False, "spare": 0, **more}


def _quantize(name, experts, rows, cols, **more):
    return {"name": name, "op": "quantize", "experts": experts, "rows": rows, "cols": cols,
            "gather": 0, "dual": True, "sums": False, "rotate": "hadamard", "spare": 0, **more}


def listed():
    return [
        # one token of one sequence through a served block's gate: latency
        _fused("fused one token", "fprop", 1, 14336, 4096, act="silu", mul=True),
        # a ragged batch with bias, the exact GELU and a float32 residual; every
        # extent ends inside a tile
        _fused("fused ragged f32", "fprop", 1237, 2081, 2080, dtype="f32", bias=True, act="gelu",
               residual=True),
        # training: a block's gate at a micro-batch's tokens, kept for backward
        _fused("fused gate 8192", "fprop", 8192, 14336, 4096, act="silu", mul=True, pre=True),
        # backward of that gate and of what it multiplies, one product for both
        _back("back gate 8192", 8192, 14336, 4096, mul=True),
        # backward of a small layer with the tanh GELU in float32
        _back("back ragged f32", 777, 1056, 992, dtype="f32", act="gelu_tanh"),
        # a served batch's 48 rows over 8 experts: latency, weights read once
        _experts("experts decode", "fprop", 8, 48, 4096, 4096, bias=True, act="silu"),
        # training: two experts a token, 8 experts at the block's width
        _experts("experts fprop", "fprop", 8, 16384, 4096, 4096, act="silu", mul=True),
        # input gradient of many small experts, with the rows' other gradient
        _experts("experts dgrad small", "dgrad", 64, 8192, 2048, 1024, residual=True, spare=100),
        # weight gradient, summed onto the last micro-batch's in float32
        _experts("experts wgrad", "wgrad", 8, 16384, 4096, 4096, dtype="f32", residual=True),
        # a served batch's rows to their experts: latency, forward only
        _quantize("quantize decode", 8, 48, 4096, gather=24, dual=False),
        # training: 8192 tokens to two experts each
        _quantize("quantize gather", 8, 16384, 4096, gather=8192),
        # the gradient of many small experts' outputs, with their biases'
        _quantize("quantize sums", 64, 8192, 1056, sums=True, rotate="none", spare=100),
    ]


def _log(rng, low, high):
    return max(low, min(high, round(2 ** rng.uniform(math.log2(low), math.log2(high)))))


def draw(rng):
    op = rng.choice(["fused", "fused", "back", "experts", "experts", "quantize"])
    if op == "quantize":
        cols = 32 * _log(rng, 4, 128)
        rows = _log(rng, 1, 16384 * 4096 // cols if cols > 4096 else 16384)
        experts = _log(rng, 1, 96)
        case = _quantize("", experts, rows, cols, gather=rng.choice([0, 0, max(1, rows // 2)]),
                         dual=rng.random() < 0.7, sums=rng.random() < 0.4,
                         rotate=rng.choice(["none", "hadamard", "hadamard", "hadamard16"]),
                         spare=rng.choice([0, 0, rows // 8]))
    else:
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
        more = {"dtype": rng.choice(["bf16", "bf16", "f32"])}
        if op == "back":
            more.update(act=act if act != "none" else "silu", mul=rng.random() < 0.5)
        k = 32 * _log(rng, 2, 256)
        n = _log(rng, 33, 8192)
        # half the largest listed product at most
        m = _log(rng, 1, min(8192, 8192 * 14336 * 2048 // (n * k)))
        if op == "back":
            case = _back("", m, n, k, **more)
        elif op == "fused":
            case = _fused("", rng.choice(["fprop", "fprop", "dgrad", "wgrad"]), m, n, k, act=act,
                          bias=rng.random() < 0.5, mul=rng.random() < 0.3,
                          residual=rng.random() < 0.5, pre=rng.random() < 0.3, **more)
        else:
            kind = rng.choice(["fprop", "fprop", "dgrad", "wgrad"])
            experts = _log(rng, 1, max(1, min(64, (1 << 28) // (n * k))))
            if kind == "fprop":
                more.update(act=act, bias=rng.random() < 0.4, mul=rng.random() < 0.3)
            case = _experts("", kind, experts, m, n, k, residual=rng.random() < 0.4,
                            spare=rng.choice([0, 0, m // 8]), **more)
    del case["name"]
    return case


# ---- inputs -----------------------------------------------------------------

def _padded(mn, k):
    return -(-mn // 256) * 256, -(-k // 128) * 128


def _scaled_blocks(y):
    """(E2M1 values, exponents) of blocks of 32 along y's last dimension."""
    mn, k = y.shape
    b = y.reshape(mn, k // 32, 32)
    amax = b.abs().amax(2)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, -127)
    t = torch.ldexp(b, -e[:, :, None]).clamp(-6, 6)
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, t).reshape(mn, k), e


def _tile_scales(e):
    mn, nkb = e.shape
    mnp, kp = _padded(mn, nkb * 32)
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, kp // 32 - nkb, 0, mnp - mn))
    return s.view(mnp // 256, 4, 4, 16, kp // 128, 4).permute(4, 0, 1, 5, 3, 2).contiguous().flatten()


def _tile_values(t):
    """[MN, K] values (one byte each) in the operand's order, padded with zeros."""
    mn, k = t.shape
    mnp, kp = _padded(mn, k)
    t = torch.nn.functional.pad(t, (0, kp - k, 0, mnp - mn))
    return t.view(mnp // 16, 16, kp // 128, 4, 32).permute(0, 2, 3, 1, 4).contiguous()


def _pack(y):
    """(codes, scales) buffers of an operand given as K-major values [MN, K]."""
    t, e = _scaled_blocks(y)
    a = t.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = _tile_values(code + 8 * torch.signbit(t).to(torch.uint8)).view(-1, 2)
    return (code[:, 0] + 16 * code[:, 1]).contiguous(), _tile_scales(e)


def _values(mn, k, gen, scale):
    """Rotated operands' values: near normal, rows and blocks of unlike sizes."""
    y = torch.randn(mn, k, generator=gen, device="cuda")
    y *= scale * torch.exp(0.5 * torch.randn(mn, 1, generator=gen, device="cuda"))
    return y


def _sizes(case, gen):
    """Rows of each expert as a router leaves them: popular and idle ones."""
    experts, rows = case["experts"], case["rows"] - case["spare"]
    liking = torch.softmax(0.8 * torch.randn(experts, generator=gen, device="cuda"), 0)
    at = torch.multinomial(liking, max(1, rows), replacement=True, generator=gen)[:rows]
    return torch.bincount(at, minlength=experts)


def _slices(rows, experts):
    """128-deep slices that hold any `experts` groups of `rows` rows together."""
    return (rows + 127 * experts) // 128


def _starts(sizes):
    """(first row, first slice) of each group, and both behind the last one."""
    zero = sizes.new_zeros(1)
    return (torch.cat([zero, sizes.cumsum(0)]), torch.cat([zero, ((sizes + 127) // 128).cumsum(0)]))


def _places(sizes, rows):
    """(group of each of `rows` rows, its place along the grouped operand's K);
    rows behind the last group have group E and place -1."""
    first, slices = _starts(sizes)
    i = torch.arange(rows, device="cuda")
    e = torch.searchsorted(first[1:].contiguous(), i, right=True)
    e1 = e.clamp(max=len(sizes) - 1)
    return e, torch.where(e < len(sizes), slices[e1] * 128 + i - first[e1], -1)


def _grouped_values(y, sizes):
    """Rows [R, C] -> K-major values [C, K] with every group's K padded to 128."""
    rows, cols = y.shape
    k = 128 * _slices(rows, len(sizes))
    place = _places(sizes, rows)[1]
    out = y.new_zeros(k + 1, cols)      # the last row takes what belongs to no group
    out.index_copy_(0, torch.where(place < 0, k, place), y)
    return out[:k].t().contiguous()


def _weights(case, gen):
    """The experts' stacked matrices as one operand [E * out, in] (fprop) or,
    transposed matrix by matrix, [in, E * out padded to 128] (dgrad)."""
    experts, n, k = case["experts"], case["n"], case["k"]
    if case["kind"] == "fprop":
        return _values(experts * n, k, gen, 0.02)
    kp = -(-k // 128) * 128
    return torch.nn.functional.pad(_values(experts * n, k, gen, 0.02), (0, kp - k)) \
        .view(experts, n, kp).transpose(0, 1).reshape(n, experts * kp).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "quantize":
        sizes = _sizes(case, gen)
        s["ends"] = sizes.cumsum(0).to(torch.int32)
        source = case["gather"] or case["rows"]
        s["x"] = rnd(source, case["cols"]).to(torch.bfloat16)
        s["index"] = (torch.randint(0, source, (case["rows"],), generator=gen, device="cuda")
                      if case["gather"] else None)
        n = 16 if case["rotate"] == "hadamard16" else 32
        s["rotation"] = torch.tensor(
            [[(-1.0) ** bin((i & j) % n).count("1") / math.sqrt(n) if i // n == j // n else 0.0
              for j in range(32)] for i in range(32)], device="cuda")
        # two E2M1 codes of a byte as two float8 values, for the outputs
        value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
        value = torch.cat([value, -value]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["pairs"] = torch.stack([value.repeat(16), value.repeat_interleave(16)], 1) \
            .contiguous().view(torch.int16).flatten()
        return s
    dt, n, k = DTYPES[case["dtype"]], case["n"], case["k"]
    grad = case["kind"] != "fprop"
    if case["op"] == "experts":
        sizes = _sizes(case, gen)
        s["ends"] = sizes.cumsum(0).to(torch.int32)
        s["sizes"] = sizes.tolist()         # a dispatch over several devices knows them
        m = case["rows"]
        if case["kind"] == "wgrad":
            s["a"] = _pack(_grouped_values(_values(m, n, gen, 1e-4), sizes))
            s["b"] = _pack(_grouped_values(_values(m, k, gen, 1.0), sizes))
            shape = (case["experts"], n, k)
        else:
            s["a"] = _pack(_values(m, k, gen, 1e-4 if grad else 1.0))
            s["b"] = _pack(_weights(case, gen))
            shape = (m, n)
        s["bias"] = rnd(case["experts"], n) if case["bias"] else None
        s["out"] = torch.zeros(shape, dtype=dt, device="cuda")
    else:
        m = case["m"]
        s["a"] = _pack(_values(m, k, gen, 1e-4 if grad else 1.0))
        s["b"] = _pack(_values(n, k, gen, 1.0 if case["kind"] == "wgrad" else 0.02))
        shape = (m, n)
        s["bias"] = rnd(n) if case.get("bias") else None
        if case["op"] == "back":
            s["pre"] = rnd(*shape).to(dt)
    s["mul"] = rnd(*shape).to(dt) if case["mul"] else None
    s["residual"] = ((1e-3 if grad else 1.0) * rnd(*shape)).to(dt) if case.get("residual") else None
    if own:
        s["qa"], s["qb"] = _handles(case, s)
    return s


# ---- the framework's calls --------------------------------------------------

def _handles(case, s):
    """The packed operands as the package's quantizers hand them out."""
    import mxfp4_microscaled_precision_amd as mx
    axes, n, k = AXES[case["kind"]], case["n"], case["k"]

    def operand(buf, axis, mn, k, **more):
        rows, cols = (mn, k) if axis == 1 else (k, mn)
        return mx.packed_operand(*buf, rows, cols, axis, rotate="hadamard", **more)

    if case["op"] != "experts":
        return operand(s["a"], axes[0], case["m"], k), operand(s["b"], axes[1], n, k)
    experts, rows = case["experts"], case["rows"]
    if case["kind"] == "wgrad":
        return (operand(s["a"], 0, n, rows, groups=experts),
                operand(s["b"], 0, k, rows, groups=experts))
    if case["kind"] == "dgrad":
        return (operand(s["a"], 1, rows, k),
                operand(s["b"], 0, n, experts * k, groups=experts, group_rows=k))
    return (operand(s["a"], 1, rows, k),
            operand(s["b"], 1, experts * n, k, groups=experts, group_rows=n))


def _own(s):
    import mxfp4_microscaled_precision_amd as mx
    case = s["case"]
    if case["op"] == "quantize":
        q = mx.quantize_grouped(s["x"], s["ends"], index=s["index"], dual=case["dual"],
                                rotate=case["rotate"], sums=case["sums"])
        out = {"axis1": _own_operand(q.q1, s)}
        if case["dual"]:
            out["axis0"] = _own_operand(q.q0, s)
        if case["sums"]:
            out["sums"] = q.sums
        return out
    if case["op"] == "back":
        return mx.linear_act_backward(s["qa"], s["qb"], s["pre"], case["act"], mul=s["mul"],
                                      out_dtype=case["dtype"])
    more = {"out_dtype": case["dtype"], "bias": s["bias"], "activation": case["act"],
            "mul": s["mul"], "residual": s["residual"]}
    if case["op"] == "fused":
        return mx.linear_fused(case["kind"], s["qa"], s["qb"], save_pre=case["pre"], **more)
    return mx.linear_grouped(case["kind"], s["qa"], s["qb"], s["ends"], out=s["out"], **more)


def _own_operand(q, s):
    codes = torch.index_select(s["pairs"], 0, q.codes.int())
    return codes.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu)


# ---- plain forms ------------------------------------------------------------

def _unpack(buf, mn, k):
    """fp32 values [MN, K] of an operand's buffers."""
    codes, scales = buf
    mnp, kp = _padded(mn, k)
    code = torch.stack([codes & 15, codes >> 4], 1).view(mnp // 16, kp // 128, 4, 16, 32)
    code = code.permute(0, 3, 1, 2, 4).reshape(mnp, kp // 32, 32)[:mn].int()
    a, m = (code & 7) >> 1, (code & 1).float()
    v = torch.where(a > 0, torch.ldexp(1 + 0.5 * m, a - 1), 0.5 * m)
    v = torch.where(code > 7, -v, v)
    e = scales.view(kp // 128, mnp // 256, 4, 4, 16, 4).permute(1, 2, 5, 4, 0, 3)
    e = e.reshape(mnp, kp // 32)[:mn].int() - 127
    return torch.ldexp(v, e[:, :, None]).reshape(mn, kp)[:, :k]


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) \
            + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _epilogue(c, bias, s, rows=slice(None)):
    """(act(c + bias) * mul + residual, c + bias)"""
    pre = c if bias is None else c + bias
    c = _act(pre, s["case"]["act"])
    if s["mul"] is not None:
        c = c * s["mul"][rows].float()
    if s["residual"] is not None:
        c = c + s["residual"][rows].float()
    return c, pre


def _run_fused(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    c = _unpack(s["a"], case["m"], case["k"]) @ _unpack(s["b"], case["n"], case["k"]).t()
    c, pre = _epilogue(c, s["bias"], s)
    return (c.to(dt), pre.to(dt)) if case["pre"] else c.to(dt)


def _run_back(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    g = _unpack(s["a"], case["m"], case["k"]) @ _unpack(s["b"], case["n"], case["k"]).t()
    pre = s["pre"].float()
    dz = g * _act_slope(pre, case["act"])
    if s["mul"] is None:
        return dz.to(dt)
    return (dz * s["mul"].float()).to(dt), (g * _act(pre, case["act"])).to(dt)


def _run_experts(s):
    case, out = s["case"], s["out"]
    n, k, rows = case["n"], case["k"], case["rows"]
    at = slot = 0
    if case["kind"] == "wgrad":
        depth = 128 * _slices(rows, case["experts"])
        a, b = _unpack(s["a"], n, depth), _unpack(s["b"], k, depth)
    elif case["kind"] == "dgrad":
        kp = -(-k // 128) * 128
        a, b = _unpack(s["a"], rows, k), _unpack(s["b"], n, case["experts"] * kp)
    else:
        a, b = _unpack(s["a"], rows, k), _unpack(s["b"], case["experts"] * n, k)
    for e, size in enumerate(s["sizes"]):
        mine = slice(at, at + size)
        if case["kind"] == "wgrad":
            deep = slice(slot * 128, slot * 128 + size)
            out[e] = _epilogue(a[:, deep] @ b[:, deep].t(), None, s, e)[0]
        elif size:
            w = b[e * n:(e + 1) * n] if case["kind"] == "fprop" else b[:, e * kp:e * kp + k]
            bias = None if s["bias"] is None else s["bias"][e]
            out[mine] = _epilogue(a[mine] @ w.t(), bias, s, mine)[0].to(out.dtype)
        at, slot = at + size, slot + -(-size // 128)
    return out


def _float_operand(y, s):
    if s["case"]["rotate"] != "none":
        y = (y.reshape(-1, 32) @ s["rotation"]).reshape(y.shape)
    t, e = _scaled_blocks(y)
    codes = _tile_values(t.to(torch.float8_e4m3fn).view(torch.uint8)).view(torch.float8_e4m3fn)
    return codes.flatten(), _tile_scales(e).view(torch.float8_e8m0fnu)


def _run_quantize(s):
    case = s["case"]
    sizes = torch.diff(s["ends"].long(), prepend=s["ends"].new_zeros(1))
    x = (s["x"] if s["index"] is None else s["x"][s["index"]]).float()
    e, place = _places(sizes, case["rows"])
    out = {"axis1": _float_operand(torch.where(place[:, None] < 0, 0.0, x), s)}
    if case["dual"]:
        out["axis0"] = _float_operand(_grouped_values(x, sizes), s)
    if case["sums"]:
        total = torch.zeros(case["experts"] + 1, case["cols"], dtype=torch.float64, device="cuda")
        out["sums"] = total.index_add_(0, e, x.double())[:-1].float()
    return out


def run(state):
    if own:
        return _own(state)
    return {"fused": _run_fused, "back": _run_back, "experts": _run_experts,
            "quantize": _run_quantize}[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    operand = 17 / 32       # bytes of an element: 4 bits, and a scale byte for 32
    if case["op"] == "quantize":
        rows, cols, live = case["rows"], case["cols"], case["rows"] - case["spare"]
        total = min(live, case["gather"] or live) * cols * 2 + case["experts"] * 4
        total += live * 8 if case["gather"] else 0
        total += math.prod(_padded(rows, cols)) * operand
        if case["dual"]:
            total += math.prod(_padded(cols, 128 * _slices(rows, case["experts"]))) * operand
        total += case["experts"] * cols * 4 if case["sums"] else 0
        turn = {"none": 0, "hadamard": 6, "hadamard16": 5}[case["rotate"]]
        return {"bytes": total, "flops": live * cols * ((2 if case["dual"] else 1) * (turn + 3)
                                                        + bool(case["sums"]))}
    wide, n, k = {"bf16": 2, "f32": 4}[case["dtype"]], case["n"], case["k"]
    if case["op"] != "experts":
        m = case["m"]
        full = 1 + sum(bool(case.get(x)) for x in ("mul", "residual", "pre"))
        if case["op"] == "back":
            full = 4 if case["mul"] else 2
        return {"bytes": (m + n) * k * operand + full * m * n * wide
                + (n * 4 if case.get("bias") else 0), "flops": 2 * m * n * k}
    live, experts = case["rows"] - case["spare"], case["experts"]
    full = 1 + sum(bool(case[x]) for x in ("mul", "residual"))
    if case["kind"] == "wgrad":
        return {"bytes": live * (n + k) * operand + full * experts * n * k * wide,
                "flops": 2 * live * n * k}
    busy = experts * (1 - (1 - 1 / experts) ** live)    # experts with any row, of as many alike
    return {"bytes": (live + busy * n) * k * operand + full * live * n * wide
            + (busy * n * 4 if case["bias"] else 0), "flops": 2 * live * n * k}


# ---- in 64 bits -------------------------------------------------------------

def _exact_values(buf, mn, k):
    """[MN, K] in 64 bits: every element's code and scale looked up by its place."""
    codes, scales = buf
    mnp, kp = _padded(mn, k)
    m = torch.arange(mn, device="cuda")[:, None]
    c = torch.arange(k, device="cuda")[None, :]
    byte = codes[((m // 16) * (kp // 128) + c // 128) * 1024 + (c % 128 // 32) * 256
                 + (m % 16) * 16 + c % 32 // 2]
    code = torch.where(c % 2 == 1, byte // 16, byte % 16).long()
    table = [0, .5, 1, 1.5, 2, 3, 4, 6]
    table = torch.tensor(table + [-v for v in table], dtype=torch.float64, device="cuda")
    b = torch.arange(k // 32, device="cuda")[None, :]
    h = m // 16 % 16
    s = scales[((b // 4) * (mnp // 256) + m // 256) * 1024 + (h // 4) * 256 + (b % 4) * 64
               + (m % 16) * 4 + h % 4]
    return table[code] * torch.exp2(s.double() - 127).repeat_interleave(32, 1)


def _exact_act(z, act):
    """(act(z), act'(z))"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # z times a logistic function of u, whose slope is du
    c = 2 * math.sqrt(2 / math.pi)
    u, du = (z, 1.0) if act == "silu" else (c * (z + 0.044715 * z ** 3),
                                            c * (1 + 0.134145 * z ** 2))
    p = torch.sigmoid(u)
    return z * p, p + z * p * (1 - p) * du


def _exact_operand(blocks, mn, k):
    """(values, scales) in their packed places of blocks [MN, K / 32, 32]."""
    mnp, kp = _padded(mn, k)
    amax = blocks.abs().max(2).values
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -1000))) - 2
    e = e.clamp(-127, 127)
    t = blocks / torch.exp2(e)[:, :, None]
    p = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -40))).clamp(min=0)
    step = torch.exp2(p - 1)
    t = (torch.round(t / step) * step).clamp(-6, 6).reshape(mn, k)
    m = torch.arange(mn, device="cuda")[:, None]
    c = torch.arange(k, device="cuda")[None, :]
    codes = torch.zeros(mnp * kp, dtype=torch.float64, device="cuda")
    where = ((m // 16) * (kp // 128) + c // 128) * 2048 + (c % 128 // 32) * 512 + (m % 16) * 32 + c % 32
    codes[where.flatten()] = t.flatten()
    b = torch.arange(k // 32, device="cuda")[None, :]
    h = m // 16 % 16
    where = ((b // 4) * (mnp // 256) + m // 256) * 1024 + (h // 4) * 256 + (b % 4) * 64 \
        + (m % 16) * 4 + h % 4
    scales = torch.full((mnp * kp // 32,), 2.0 ** -127, dtype=torch.float64, device="cuda")
    scales[where.flatten()] = torch.exp2(e).flatten()
    return codes, scales


def _exact_quantize(case, s):
    ends = s["ends"].tolist()
    live, cols = ends[-1], case["cols"]
    x = s["x"].double() if s["index"] is None else s["x"].double()[s["index"]]
    h = s["rotation"].double()
    if case["rotate"] != "none":
        h = torch.sign(h) / math.sqrt(16 if case["rotate"] == "hadamard16" else 32)
    turned = (lambda b: b) if case["rotate"] == "none" else (lambda b: b @ h)
    rows = torch.zeros(case["rows"], cols, dtype=torch.float64, device="cuda")
    rows[:live] = x[:live]
    out = {"axis1": _exact_operand(turned(rows.view(-1, cols // 32, 32)), *rows.shape)}
    deep = torch.zeros(cols, 128 * _slices(case["rows"], case["experts"]), dtype=torch.float64,
                       device="cuda")
    sums = torch.zeros(case["experts"], cols, dtype=torch.float64, device="cuda")
    at = slot = 0
    for e, end in enumerate(ends):
        deep[:, slot * 128:slot * 128 + end - at] = x[at:end].t()
        sums[e] = x[at:end].sum(0)
        at, slot = end, slot + (end - at + 127) // 128
    if case["dual"]:
        out["axis0"] = _exact_operand(turned(deep.view(cols, -1, 32)), *deep.shape)
    if case["sums"]:
        out["sums"] = sums
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(case, s)
    n, k = case["n"], case["k"]
    wide = {x: s[x].double() for x in ("bias", "mul", "residual", "pre") if s.get(x) is not None}
    if case["op"] != "experts":
        c = _exact_values(s["a"], case["m"], k) @ _exact_values(s["b"], n, k).t()
        if case["op"] == "back":
            y, slope = _exact_act(wide["pre"], case["act"])
            return (c * slope * wide["mul"], c * y) if case["mul"] else c * slope
        pre = c + wide.get("bias", 0.0)
        y = _exact_act(pre, case["act"])[0] * wide.get("mul", 1.0) + wide.get("residual", 0.0)
        return (y, pre) if case["pre"] else y
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    experts, rows, ends = case["experts"], case["rows"], s["ends"].tolist()
    depth = 128 * _slices(rows, experts)
    kp = -(-k // 128) * 128
    if case["kind"] == "wgrad":
        a, b = _exact_values(s["a"], n, depth), _exact_values(s["b"], k, depth)
    else:
        a = _exact_values(s["a"], rows, k)
        b = _exact_values(s["b"], *((experts * n, k) if case["kind"] == "fprop"
                                    else (n, experts * kp)))
    at = slot = 0
    for e, end in enumerate(ends):
        if case["kind"] == "wgrad":
            last = slot + (end - at + 127) // 128
            out[e] = a[:, slot * 128:last * 128] @ b[:, slot * 128:last * 128].t()
            slot = last
        elif end > at:
            w = b.view(experts, n, k)[e] if case["kind"] == "fprop" \
                else b.view(n, experts, kp)[:, e, :k]
            out[at:end] = a[at:end] @ w.t() + (wide["bias"][e] if case["bias"] else 0.0)
        at = end
    out = _exact_act(out, case["act"])[0] * wide.get("mul", 1.0) + wide.get("residual", 0.0)
    if case["kind"] != "wgrad":
        out[at:] = 0        # rows of no expert stay as they were
    return out
