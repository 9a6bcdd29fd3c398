"""The grouped quantizer against the oracle, bit for bit."""
import numpy as np
import pytest

import oracle
from datagen import activations_bf16
from gpu_util import host_u8, to_dev, to_dev_strided

pytestmark = pytest.mark.gpu

SIZES = [0, 1, 31, 32, 33, 0, 127, 128, 129, 300]


def _ends(sizes):
    import torch
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")


def _check(q, x, ranges, group_rows, rotate, rnd, seeds, dual=True):
    rows, cols = x.shape
    slices = oracle.grouped_slices_ref(rows, len(ranges), group_rows)
    one, zero = oracle.grouped_quantize_ref(x, ranges, slices, rotate, rnd, *seeds)
    for got, ref, what in ((q.q1, one, "axis 1"), (q.q0, zero, "grouped axis 0")):
        if got is None:
            assert not dual
            continue
        codes, scales = host_u8(got.codes), host_u8(got.scales)
        assert np.array_equal(scales, ref[1]), f"{what}: {np.count_nonzero(scales != ref[1])} scales"
        assert np.array_equal(codes, ref[0]), f"{what}: {np.count_nonzero(codes != ref[0])} code bytes"
        assert (got.groups, got.group_rows) == (len(ranges), group_rows)


@pytest.mark.parametrize("rnd", ["rne", "sr"])
@pytest.mark.parametrize("rotate", ["none", "hadamard", "rand_sign_hadamard", "hadamard16"])
@pytest.mark.parametrize("cols", [32, 416])
def test_ragged_groups(mx, cols, rotate, rnd):
    rng = np.random.Generator(np.random.PCG64(cols))
    rows = sum(SIZES) + 37                            # some in no group
    x = activations_bf16(rng, (rows, cols), outlier_frac=0.01)
    q = mx.quantize_grouped(to_dev(x), _ends(SIZES), rotate=rotate, round=rnd, seed1=5, seed0=9)
    _check(q, x, oracle.group_ranges_ref(np.cumsum(SIZES), rows), -1, rotate, rnd, (5, 9))


@pytest.mark.parametrize("sizes,spare", [([1], 0), ([0, 0, 7], 0), ([0], 5), ([255, 1], 0),
                                         ([128, 128], 128), ([1] * 150, 3), ([0] * 64 + [40], 0)])
@pytest.mark.parametrize("dual", [True, False])
def test_sizes_of_groups(mx, sizes, spare, dual):
    rng = np.random.Generator(np.random.PCG64(len(sizes)))
    rows = sum(sizes) + spare
    x = activations_bf16(rng, (rows, 160), outlier_frac=0.01)
    q = mx.quantize_grouped(to_dev(x), _ends(sizes), dual=dual, sums=True)
    ranges = oracle.group_ranges_ref(np.cumsum(sizes), rows)
    _check(q, x, ranges, -1, "hadamard", "rne", (0, 0), dual)
    _check_sums(q.sums, x, ranges)


def _check_sums(sums, x, ranges):
    """n terms are added with at most 5 + n / 128 + 3 roundings each (32 by
    halves, then a quarter of the blocks in a row, then four)."""
    v = (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    got = sums.double().cpu().numpy()
    for e, (a, b) in enumerate(ranges):
        bound = (9 + (b - a) / 128) * 2.0 ** -24 * np.abs(v[a:b]).sum(0)
        assert np.all(np.abs(got[e] - v[a:b].sum(0)) <= bound), f"sums of group {e}"


@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("dual", [True, False])
def test_gathered_rows(mx, bits, dual):
    """The router's order: rows that come up twice, none (-1) and outside."""
    import torch
    rng = np.random.Generator(np.random.PCG64(bits))
    src = activations_bf16(rng, (90, 96), outlier_frac=0.01)
    index = rng.integers(0, 90, 260)
    index[[3, 100, 259]] = -1
    index[[7, 130]] = 90
    if bits == 64:
        index[9] = 1 << 32
    x = np.where(((index >= 0) & (index < 90))[:, None], src[np.clip(index, 0, 89)], 0)
    sizes = [100, 0, 31, 120]
    for source in (to_dev(src), to_dev_strided(src, 104)):
        q = mx.quantize_grouped(source, _ends(sizes), sums=True, dual=dual, round="sr", seed1=3,
                                seed0=4, index=torch.tensor(index, device="cuda").to(
                                    torch.int32 if bits == 32 else torch.int64))
        ranges = oracle.group_ranges_ref(np.cumsum(sizes), 260)
        _check(q, x.astype(np.uint16), ranges, -1, "hadamard", "sr", (3, 4), dual)
        _check_sums(q.sums, x.astype(np.uint16), ranges)


@pytest.mark.parametrize("shape", [(1, 33, 32), (3, 128, 160), (5, 96, 64), (4, 1, 64), (2, 300, 96)])
@pytest.mark.parametrize("rotate", ["hadamard", "rand_sign_hadamard"])
def test_stacked_matrices(mx, shape, rotate):
    rng = np.random.Generator(np.random.PCG64(shape[1]))
    e, r, c = shape
    x = activations_bf16(rng, (e * r, c), outlier_frac=0.01)
    q = mx.quantize_grouped(to_dev(x).view(shape), rotate=rotate, seed1=2, seed0=2, sums=True)
    ranges = [(i * r, (i + 1) * r) for i in range(e)]
    _check(q, x, ranges, r, rotate, "rne", (2, 2))
    _check_sums(q.sums, x, ranges)


@pytest.mark.parametrize("ends", [[50, 20, 300, 200, 400], [-5, -1, 0, 7, 7], [400, 0, 0, 0, 0],
                                  [2 ** 31 - 1, -2 ** 31, 5, 6, 7]])
def test_ends_out_of_order(mx, ends):
    """An end below an earlier one is an empty group, one past the rows their end."""
    import torch
    rng = np.random.Generator(np.random.PCG64(8))
    x = activations_bf16(rng, (310, 64), outlier_frac=0.01)
    q = mx.quantize_grouped(to_dev(x), torch.tensor(ends, dtype=torch.int32, device="cuda"),
                            sums=True)
    ranges = oracle.group_ranges_ref(ends, 310)
    _check(q, x, ranges, -1, "hadamard", "rne", (0, 0))
    _check_sums(q.sums, x, ranges)


def test_nonfinite_rows_mark_their_own_group(mx):
    """NaN and Inf next to a border: the neighbouring group's blocks stay clean."""
    rng = np.random.Generator(np.random.PCG64(6))
    x = activations_bf16(rng, (100, 64), outlier_frac=0.0)
    x[39, 3], x[40, 50] = 0x7FC0, 0xFF80
    ranges = oracle.group_ranges_ref([40, 41, 90], 100)
    q = mx.quantize_grouped(to_dev(x), _ends([40, 1, 49]))
    _check(q, x, ranges, -1, "hadamard", "rne", (0, 0))


def test_empty(mx):
    import torch
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    q = mx.quantize_grouped(x, _ends([0, 0]), sums=True)
    assert q.q1.codes.numel() == q.q0.codes.numel() == 0 and not q.sums.any()
    assert (q.q0.axis, q.q0.mn) == (mx.AXIS_GROUPED, 64)
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    q = mx.quantize_grouped(x, _ends([0]), index=torch.empty(0, dtype=torch.int64, device="cuda"))
    assert q.q1.codes.numel() == 0
    q = mx.quantize_grouped(torch.empty((3, 0), dtype=torch.bfloat16, device="cuda"), _ends([1, 2]),
                            sums=True)
    assert q.sums.shape == (2, 0)


def test_no_source_rows(mx):
    """An index into nothing: rows of zeros."""
    import torch
    x = torch.empty((0, 96), dtype=torch.bfloat16, device="cuda")
    for dual in (True, False):
        q = mx.quantize_grouped(x, _ends([3, 150]), sums=dual, dual=dual,
                                index=torch.arange(200, device="cuda", dtype=torch.int32))
        _check(q, np.zeros((200, 96), np.uint16), oracle.group_ranges_ref([3, 153], 200), -1,
               "hadamard", "rne", (0, 0), dual)
        assert not dual or not q.sums.any()


def test_same_bytes_as_the_single_quantizers(mx):
    """Groups of whole slices: the dual quantizer's operands, slice by slice."""
    rng = np.random.Generator(np.random.PCG64(12))
    x = to_dev(activations_bf16(rng, (512, 288), outlier_frac=0.01))
    q = mx.quantize_grouped(x, _ends([512]), seed1=1, seed0=2)
    one, zero = mx.quantize_dual(x, seed1=1, seed0=2)
    n = zero.codes.numel()
    assert np.array_equal(host_u8(q.q1.codes), host_u8(one.codes))
    assert np.array_equal(host_u8(q.q1.scales), host_u8(one.scales))
    assert q.q0.codes.numel() == n // 4 * 4 and np.array_equal(host_u8(q.q0.codes), host_u8(zero.codes))
