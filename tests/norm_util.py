"""Helpers shared by the norm, gradient and clipping tests."""
import numpy as np

import oracle
from datagen import bf16_bits_to_f32, f32_to_bf16_bits


def values(rng, shape, bf16, scale=1.0):
    """Normal values (one column in sixteen 30 times larger) as fp32, already
    rounded to bf16 where the tensor is."""
    v = rng.standard_normal(shape).astype(np.float32) * np.float32(scale)
    if len(shape) == 2 and shape[1] >= 16:
        v[:, rng.integers(0, shape[1], shape[1] // 16)] *= np.float32(30)
    return bf16_bits_to_f32(f32_to_bf16_bits(v)) if bf16 else v


def dev(v, bf16, ld=None, fill=float("nan")):
    """fp32 array -> CUDA tensor; with ld a row-strided view whose padding
    holds `fill`."""
    import torch
    t = torch.from_numpy(np.array(v, dtype=np.float32, copy=True))
    t = t.to(torch.bfloat16 if bf16 else torch.float32)
    if ld is not None:
        big = torch.full((v.shape[0], ld), fill, dtype=t.dtype)
        big[:, :v.shape[1]] = t
        return big.cuda()[:, :v.shape[1]]
    return t.cuda()


def host(t):
    return t.detach().float().cpu().numpy()


def operand_ref(y, axis, rotate, rnd, seed, fmt):
    """(codes, scales) buffers of the operand of y."""
    q = oracle.quantize_values_ref(y, axis, rotate=rotate, rounding=rnd, seed=seed, fmt=fmt)
    tile = oracle.tile_codes_fp8 if fmt == "fp8_e4m3" else oracle.tile_codes
    return tile(q.codes), oracle.tile_scales(q.scales, q.codes.shape[1])


def check_operand(q, y, axis, rotate, rnd, seed, fmt, what):
    codes, scales = operand_ref(y, axis, rotate, rnd, seed, fmt)
    got_s, got_c = q.scales.cpu().numpy(), q.codes.cpu().numpy()
    assert np.array_equal(got_s, scales), f"{what}: {np.count_nonzero(got_s != scales)} scales differ"
    assert np.array_equal(got_c, codes), f"{what}: {np.count_nonzero(got_c != codes)} code bytes differ"
    assert (q.desc.rows, q.desc.cols, q.desc.axis) == (*y.shape, axis)
    assert q.format == fmt
