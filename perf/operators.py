"""Cases and plain forms of the operators around the quantized linears.

A training step with MXFP4 linears spends the rest of a layer's time in the
tensors between them. Three operators cover that:

  norm   h = x + residual; y = h * rstd * weight with rstd = 1 / sqrt(mean(h^2)
         + eps) per row; y rotated and quantized into the packed operands the
         linears read (axis 1 for the forward product and, in training, axis 0
         for the weight gradient).
  grad   the norm's backward pass: the gradient of h (plus the gradient that
         arrives through the residual path) and of the weight.
  clip   the global 2-norm over many gradient tensors, and the gradients
         scaled so that it does not exceed max_norm.

`run` computes them from elementary torch operations; with `own` set it calls
the package's entry points. The operand buffers are compared in their packed
tile order: E4M3 codes as the float8 values they are, E2M1 codes unpacked into
float8 values (which hold every E2M1 value), scales as float8_e8m0fnu.
"""
import math

import torch

own = False

EPS = 1e-5
CLIP_EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# largest exponent of an element format, and its largest value
TOP = {"fp8_e4m3": (8, 448.0), "fp4_e2m1": (2, 6.0)}


def _norm(name, rows, cols, **more):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": "bf16",
            "weight": "bf16", "residual": True, "dual": False, "format": "fp8_e4m3",
            "rotate": "hadamard", **more}


def _grad(name, rows, cols, **more):
    return {"name": name, "op": "grad", "rows": rows, "cols": cols, "dtype": "bf16",
            "weight": "bf16", "residual": True, **more}


def _clip(name, layers, d, kv, ff, **more):
    return {"name": name, "op": "clip", "layers": layers, "d": d, "kv": kv, "ff": ff,
            "dtype": "f32", "align": 64, "max_norm": 1.0, **more}


def listed():
    return [
        # one token of one sequence on its way through a served layer: latency
        _norm("norm one token", 1, 4096),
        # a ragged batch of tokens over a float32 residual stream, first layer
        # (no branch to add yet), a width that ends inside a 128-wide tile
        _norm("norm ragged f32", 1237, 2080, dtype="f32", weight="f32", residual=False,
              rotate="none"),
        # the tokens of one forward-only step at the block's width
        _norm("norm forward 8192", 8192, 4096),
        # training, both orientations in MXFP4: a smaller micro-batch
        _norm("norm train fp4", 4096, 4096, dual=True, format="fp4_e2m1"),
        # training, both orientations, the block's tokens and width
        _norm("norm train 16384", 16384, 4096, dual=True),
        # backward at the block's tokens and width, with the residual path
        _grad("grad 16384", 16384, 4096),
        # backward of a ragged batch in float32, no residual path
        _grad("grad ragged f32", 777, 1056, dtype="f32", weight="f32", residual=False),
        # backward of a small micro-batch: latency
        _grad("grad small", 32, 512),
        # one block's nine gradients as the weight-gradient product leaves them
        _clip("clip block f32", 1, 4096, 1024, 14336),
        # a deep, narrow model's bf16 gradients, packed one after the other
        # without padding: hundreds of tensors, few of them aligned
        _clip("clip many bf16", 32, 517, 129, 1811, dtype="bf16", align=1, max_norm=0.25),
        # a tiny model below the limit: latency, nothing to scale
        _clip("clip tiny", 1, 256, 64, 704),
    ]


def draw(rng):
    op = rng.choice(["norm", "norm", "grad", "clip"])
    if op == "clip":
        layers = round(2 ** rng.uniform(0, 5))
        # layers * 14.5 d^2 parameters at most: within the largest listed case
        d = round(2 ** rng.uniform(6, math.log2(3800 / math.sqrt(layers))))
        case = _clip("", layers, d, max(1, d // rng.choice([1, 2, 4])), round(d * 3.5),
                     dtype=rng.choice(["f32", "bf16"]), align=rng.choice([1, 64]),
                     max_norm=2.0 ** rng.randint(-4, 2))
    else:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        cols = 32 * round(2 ** rng.uniform(2, 8.5))
        most = 16384 * 4096 // (cols * (2 if dtype == "f32" else 1))
        rows = round(2 ** rng.uniform(0, math.log2(min(16384, most))))
        more = {"dtype": dtype, "weight": rng.choice(["bf16", "f32"]),
                "residual": rng.random() < 0.7}
        if op == "norm":
            dual = rng.random() < 0.5
            rows = max(32, rows // 32 * 32) if dual else rows
            case = _norm("", rows, cols, dual=dual, **more,
                         format=rng.choice(["fp8_e4m3", "fp8_e4m3", "fp4_e2m1"]),
                         rotate=rng.choice(["hadamard", "none", "hadamard16"]))
        else:
            case = _grad("", rows, cols, **more)
    del case["name"]
    return case


def _shapes(case):
    """Gradient shapes of `layers` blocks: q, k, v, o, gate, up, down and two
    norm weights each; the vectors are float32."""
    d, kv, ff = case["d"], case["kv"], case["ff"]
    block = [(d, d), (kv, d), (kv, d), (d, d), (ff, d), (ff, d), (d, ff), (d,), (d,)]
    return block * case["layers"]


def _sizes(case):
    """(elements of the matrices, of the vectors), padding left out."""
    n = [math.prod(s) for s in _shapes(case)]
    v = sum(k for k, s in zip(n, _shapes(case)) if len(s) == 1)
    return sum(n) - v, v


def _gradient(shape, gen):
    """1e-4 times Student-t with three degrees of freedom."""
    z = torch.randn((4, *shape), generator=gen, device="cuda")
    return 1e-4 * z[0] / z[1:].square_().mean(0).sqrt_()


def _activation(rows, cols, gen):
    """N(0, 1) with one channel in a thousand 50 times larger."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    n = round(cols / 1000)
    if n:
        at = torch.randperm(cols, generator=gen, device="cuda")[:n]
        x[:, at] *= 50
    return x


def _hadamard(kind):
    """The rotation of one 32-element block as a matrix."""
    n = 16 if kind == "hadamard16" else 32
    m = [[(-1.0) ** bin(i & j).count("1") if i // n == j // n else 0.0 for j in range(32)]
         for i in range(32)]
    return torch.tensor(m, dtype=torch.float64, device="cuda") / math.sqrt(n)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "clip":
        shapes = _shapes(case)
        kinds = ["f32" if len(x) == 1 else case["dtype"] for x in shapes]
        at, ends = [], {"f32": 0, "bf16": 0}
        for shape, kind in zip(shapes, kinds):
            at.append(ends[kind])
            ends[kind] += -(-math.prod(shape) // case["align"]) * case["align"]
        ins, outs = {}, {}
        for kind, n in ends.items():
            ins[kind] = _gradient((n,), gen).to(DTYPES[kind])
            outs[kind] = torch.zeros(n, dtype=DTYPES[kind], device="cuda")
        view = lambda flat: [flat[k][a:a + math.prod(x)].view(x)  # noqa: E731
                             for k, a, x in zip(kinds, at, shapes)]
        s["grads"], s["out"], s["flat"] = view(ins), view(outs), outs
        s["max_norm"] = case["max_norm"]
        if own:  # the list of gradient buffers that a training program makes once
            import mxfp4_microscaled_precision_amd as mx
            s["grad_set"], s["out_set"] = mx.GradSet(s["grads"]), mx.GradSet(s["out"])
        return s
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    weight = 1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")
    s["weight"] = weight.to(DTYPES[case["weight"]])
    if case["op"] == "norm":
        s["x"] = _activation(rows, cols, gen).to(dt)
        s["residual"] = _activation(rows, cols, gen).to(dt) if case["residual"] else None
        s["rotation"] = _hadamard(case["rotate"]).float()
        # two E2M1 codes of a byte as two float8 values, for the outputs
        value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
        value = torch.cat([value, -value]).to(torch.float8_e4m3fn).view(torch.uint8)
        pair = torch.stack([value.repeat(16), value.repeat_interleave(16)], 1).contiguous()
        s["pairs"] = pair.view(torch.int16).flatten()
    else:
        s["dy"] = _gradient((rows, cols), gen).to(dt)
        s["dres"] = _gradient((rows, cols), gen).to(dt) if case["residual"] else None
        s["h"] = _activation(rows, cols, gen).to(dt)
        s["rstd"] = (s["h"].double().square().mean(1) + EPS).rsqrt().float()
    return s


def _operand(y, case, rotation):
    """(codes, scales) of the packed operand of y [MN, K]."""
    top, largest = TOP[case["format"]]
    mn, k = y.shape
    b = y.reshape(mn, k // 32, 32)
    if case["rotate"] != "none":
        b = b @ rotation
    amax = b.abs().amax(2)
    e = (torch.frexp(amax).exponent - 1 - top).clamp(-127, 127)
    e = torch.where(amax > 0, e, -127)
    t = torch.ldexp(b, -e[:, :, None]).clamp(-largest, largest)
    if case["format"] == "fp4_e2m1":
        a = t.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        t = torch.copysign(torch.round(a / step) * step, t)
    codes = t.to(torch.float8_e4m3fn).view(torch.uint8).reshape(mn, k)
    mnp, kp = -(-mn // 256) * 256, -(-k // 128) * 128
    codes = torch.nn.functional.pad(codes, (0, kp - k, 0, mnp - mn))
    # E4M3 tiles hold 16-element chunks of their 16 rows, E2M1 tiles 32-element ones
    chunk = 32 if case["format"] == "fp4_e2m1" else 16
    codes = codes.view(mnp // 16, 16, kp // 128, 128 // chunk, chunk).permute(0, 2, 3, 1, 4)
    scales = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, (kp - k) // 32, 0, mnp - mn))
    scales = scales.view(mnp // 256, 4, 4, 16, kp // 128, 4).permute(4, 0, 1, 5, 3, 2)
    return (codes.contiguous().view(torch.float8_e4m3fn).flatten(),
            scales.contiguous().view(torch.float8_e8m0fnu).flatten())


def _run_norm(s):
    case = s["case"]
    h = s["x"]
    if s["residual"] is not None:
        h = (s["x"].float() + s["residual"].float()).to(h.dtype)  # the stream as it is stored
    hf = h.float()
    # in 64 bits: y decides values next to a rounding border
    rstd = (hf.double().square().mean(1) + EPS).rsqrt().float()
    y = hf * rstd[:, None] * s["weight"].float()
    out = {"h": h, "rstd": rstd, "axis1": _operand(y, case, s["rotation"])}
    if case["dual"]:
        out["axis0"] = _operand(y.t(), case, s["rotation"])
    return out


def _run_grad(s):
    xhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    dxhat = dy * s["weight"].float()
    dh = (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return {"dh": dh.to(s["dy"].dtype), "dweight": (dy * xhat).sum(0)}


def _run_clip(s):
    squares = torch.stack([g.float().square().sum() for g in s["grads"]])
    norm = squares.double().sum().sqrt().float()
    coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1)
    [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["out"])]
    return {"norm": norm, **s["flat"]}


def _own_operand(q, s):
    fp4 = s["case"]["format"] == "fp4_e2m1"
    codes = torch.index_select(s["pairs"], 0, q.codes.int()) if fp4 else q.codes
    if s["case"]["rotate"] == "hadamard16":
        # _hadamard negates the second half of a block after its 16-point
        # rotation, the package does not: the values come in _hadamard's signs
        # (eight of them at a time: the sign bits of half the words)
        words = codes.view(torch.int64)
        half = words.view(-1, 4)[:, 2:] if fp4 else words.view(-1, 8, 32)[:, 1::2]
        half.bitwise_xor_(-0x7F7F7F7F7F7F7F80)
    return codes.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu)


def _own_norm(s):
    import mxfp4_microscaled_precision_amd as mx
    case = s["case"]
    r = mx.rmsnorm_quantize(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                            format=case["format"], dual=case["dual"], rotate=case["rotate"])
    out = {"h": r.h, "rstd": r.rstd, "axis1": _own_operand(r.q1, s)}
    if case["dual"]:
        out["axis0"] = _own_operand(r.q0, s)
    return out


def _own_grad(s):
    import mxfp4_microscaled_precision_amd as mx
    dh, dweight = mx.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["weight"], dres=s["dres"])
    return {"dh": dh, "dweight": dweight}


def _own_clip(s):
    import mxfp4_microscaled_precision_amd as mx
    norm = mx.clip_grad_norm(s["grad_set"], s["max_norm"], out=s["out_set"])
    return {"norm": norm, **s["flat"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "grad": _own_grad, "clip": _own_clip}[op](state)
    return {"norm": _run_norm, "grad": _run_grad, "clip": _run_clip}[op](state)


def work(case):
    wide = {"bf16": 2, "f32": 4}
    if case["op"] == "clip":
        m, v = _sizes(case)
        # a square and a sum for the norm, a product for the scaling
        return {"bytes": 2 * (m * wide[case["dtype"]] + v * 4) + 4, "flops": 3 * (m + v)}
    rows, cols, w = case["rows"], case["cols"], wide[case["dtype"]]
    n = rows * cols
    small = cols * wide[case["weight"]] + rows * 4
    if case["op"] == "grad":
        return {"bytes": n * w * (4 if case["residual"] else 3) + small + cols * 4,
                "flops": 11 * n}
    total = n * w * (3 if case["residual"] else 1) + small
    bits = 8 if case["format"] == "fp8_e4m3" else 4
    turn = {"none": 0, "hadamard": 6, "hadamard16": 5}[case["rotate"]]
    shapes = [(rows, cols), (cols, rows)] if case["dual"] else [(rows, cols)]
    for mn, k in shapes:
        total += (-(-mn // 256) * 256) * (-(-k // 128) * 128) * (bits / 8 + 1 / 32)
    return {"bytes": total, "flops": n * (5 + len(shapes) * (turn + 3))}


def _exact_operand(y, case):
    """The packed operand of y [MN, K] in 64 bits, placed element by element."""
    fmt = case["format"]
    mn, k = y.shape
    mnp, kp = -(-mn // 256) * 256, -(-k // 128) * 128
    blocks = y.reshape(-1, 32)
    if case["rotate"] != "none":
        blocks = blocks @ _hadamard(case["rotate"])
    amax = blocks.abs().max(1).values
    top = 8 if fmt == "fp8_e4m3" else 2
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -1000))) - top
    e = e.clamp(-127, 127)
    t = blocks / torch.exp2(e)[:, None]
    # an element's grid: 2^-3 of its power of two (E4M3) or 2^-1 (E2M1), no
    # finer than the smallest normal number's
    low, bits, most = (-6, 3, 448.0) if fmt == "fp8_e4m3" else (0, 1, 6.0)
    p = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -40))).clamp(min=low)
    step = torch.exp2(p - bits)
    t = (torch.round(t / step) * step).clamp(-most, most).reshape(mn, k)
    m = torch.arange(mn, device="cuda")[:, None]
    c = torch.arange(k, device="cuda")[None, :]
    chunk = 16 if fmt == "fp8_e4m3" else 32
    where = ((m // 16) * (kp // 128) + c // 128) * 2048 + (c % 128 // chunk) * 16 * chunk \
        + (m % 16) * chunk + c % chunk
    codes = torch.zeros(mnp * kp, dtype=torch.float64, device="cuda")
    codes[where.flatten()] = t.flatten()
    b = torch.arange(k // 32, device="cuda")[None, :]
    g = m // 16 % 16
    where = ((b // 4) * (mnp // 256) + m // 256) * 1024 + (g // 4) * 256 + (b % 4) * 64 \
        + (m % 16) * 4 + g % 4
    scales = torch.full((mnp * kp // 32,), 2.0 ** -127, dtype=torch.float64, device="cuda")
    scales[where.flatten()] = torch.exp2(e)
    return codes, scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        total = sum(float((g.double() ** 2).sum()) for g in s["grads"])
        norm = math.sqrt(total)
        scale = min(1.0, case["max_norm"] / (norm + CLIP_EPS))
        out = {k: torch.zeros_like(f, dtype=torch.float64) for k, f in s["flat"].items()}
        for g, o in zip(s["grads"], s["out"]):
            flat = out["f32" if o.dtype == torch.float32 else "bf16"]
            flat[o.storage_offset():o.storage_offset() + o.numel()] = g.double().flatten() * scale
        return {"norm": norm, **out}
    w = s["weight"].double()
    if case["op"] == "grad":
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()
        dot = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
        dot += torch.linalg.vecdot(dy * w, h) * r ** 3 / case["cols"]
        dh = dy * w * r[:, None] - h * dot[:, None]
        if s["dres"] is not None:
            dh = dh + s["dres"].double()
        return {"dh": dh, "dweight": torch.mv((dy * h).t(), r)}
    h = s["x"].double()
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(s["x"].dtype).double()
    rstd = 1 / torch.sqrt(torch.linalg.vecdot(h, h) / case["cols"] + EPS)
    y = h * rstd[:, None] * w
    out = {"h": h, "rstd": rstd, "axis1": _exact_operand(y, case)}
    if case["dual"]:
        out["axis0"] = _exact_operand(y.t().contiguous(), case)
    return out
