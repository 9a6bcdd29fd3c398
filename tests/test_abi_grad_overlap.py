"""Memory that two gradient tensors share is refused on the host, whatever
their gaps: clipping would scale such elements once or twice, by chance. No
GPU; the addresses are never touched."""
import ctypes
import random

import numpy as np
import pytest
import torch  # noqa: F401  (the library must bind to torch's HIP runtime)

import mxfp4_microscaled_precision_amd as mx

P = 1 << 20         # a fake, aligned address
SIZE = {0: 4, 1: 2}


@pytest.fixture(scope="module")
def lib():
    return mx.load_library()


def _fill(lib, entries):
    """(status, set, what it borrows) of entries (data, rows, cols, ld, dtype)."""
    g = (mx.GradDesc * len(entries))(*[mx.GradDesc(*e) for e in entries])
    need = ctypes.c_size_t()
    assert lib.mx_grad_set_size(len(entries), g, ctypes.byref(need)) == 0
    s = mx.GradSetDesc()
    host = np.zeros(need.value // 8, np.uint64)
    st = lib.mx_grad_set_fill(len(entries), g, host.ctypes.data, need.value, ctypes.byref(s))
    return st, s, (host, g)


def _bytes(e):
    """The bytes of an entry, one by one."""
    data, rows, cols, ld, dtype = e
    n = SIZE[dtype]
    return {data + (r * ld + c) * n + k for r in range(rows) for c in range(cols) for k in range(n)}


SETS = [
    (-4, [(P, 8, 10, 20, 0), (P + 20, 8, 10, 20, 0)]),          # buf[:, :10], buf[:, 5:15]
    (-4, [(P, 8, 20, 20, 0), (P, 8, 5, 20, 0)]),                # buf, buf[:, :5]
    (-4, [(P, 8, 5, 20, 0), (P, 8, 20, 20, 0)]),
    (-4, [(P + 80, 1, 20, 20, 0), (P, 8, 5, 20, 0)]),           # buf[1], buf[:, :5]
    (0, [(P + 80 + 20, 1, 15, 15, 0), (P, 8, 5, 20, 0)]),       # buf[1, 5:], buf[:, :5]
    (-4, [(P + 80 + 20, 1, 16, 16, 0), (P, 8, 5, 20, 0)]),      # one element more
    (0, [(P, 8, 10, 20, 0), (P + 40, 8, 10, 20, 0)]),           # buf[:, :10], buf[:, 10:]
    (0, [(P, 4, 20, 40, 0), (P + 80, 4, 20, 40, 0)]),           # buf[::2], buf[1::2]
    (-4, [(P, 4, 20, 40, 0), (P + 80, 2, 20, 80, 0), (P + 80, 2, 10, 20, 0)]),
    (0, [(P, 4, 20, 40, 0), (P + 80, 2, 20, 80, 0)]),           # buf[::2], buf[1::4]
    (-4, [(P, 4, 20, 40, 0), (P + 160, 2, 20, 80, 0)]),         # buf[::2], buf[2::4]
    (0, [(P, 9, 1, 2, 0), (P + 4, 9, 1, 2, 0)]),                # two strided vectors
    (-4, [(P, 9, 1, 2, 0), (P + 4, 6, 1, 3, 0)]),               # every second, every third
    (-4, [(P, 9, 1, 2, 0), (P + 2, 9, 1, 4, 1)]),               # the half of an element
    (0, [(P, 9, 1, 2, 0), (P + 4, 9, 1, 4, 1)]),
    (0, [(P, 1 << 20, 1, 1 << 30, 0), (P + 4, 1 << 20, 1, 1 << 30, 0)]),
    (-4, [(P, 1 << 20, 1, 1 << 30, 0), (P + (((1 << 20) - 1) << 32), 1, 1, 1, 0)]),
    (0, [(P, 1 << 20, 1, 1 << 30, 0), (P + (((1 << 20) - 1) << 32) + 4, 1, 1, 1, 0)]),
]


@pytest.mark.parametrize("want,entries", SETS)
def test_within_a_set(lib, want, entries):
    assert _fill(lib, entries)[0] == want
    assert _fill(lib, entries[::-1])[0] == want


def _random_entries(rng, n):
    out = []
    for _ in range(n):
        dtype = rng.randrange(2)
        rows, cols = rng.randint(1, 6), rng.randint(1, 5)
        ld = cols + rng.choice([0, 0, 1, 2, 5, 9])
        out.append((P + rng.randrange(60) * 4, rows, cols, ld, dtype))
    return out


def test_within_a_set_against_enumeration(lib):
    """Random small tensors against their bytes one by one."""
    rng = random.Random(3)
    seen = {0: 0, -4: 0}
    for _ in range(4000):
        entries = _random_entries(rng, rng.choice([2, 2, 2, 3]))
        b = [_bytes(e) for e in entries]
        want = -4 if any(b[i] & b[j] for i in range(len(b)) for j in range(i)) else 0
        assert _fill(lib, entries)[0] == want, entries
        seen[want] += 1
    assert min(seen.values()) > 400, seen
