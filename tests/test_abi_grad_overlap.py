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


def _clip(lib, a, b):
    """Status of clipping set a into set b with a misaligned norm, which is
    refused (-3) after the sets and before anything is launched."""
    sets = []
    for entries in (a, b):
        st, s, borrowed = _fill(lib, entries)
        assert st == 0
        s.table = P
        sets.append((s, borrowed))
    (x, _), (y, _) = sets
    return lib.mx_grad_clip(ctypes.byref(x), ctypes.byref(y), 1.0, P + 2, P,
                            lib.mx_grad_workspace(), None)


FAR = P + (1 << 24)
PAIRS = [
    (-3, [(P, 8, 5, 20, 0)], [(P, 8, 5, 20, 0)]),               # in place
    (-3, [(P, 8, 5, 20, 0)], [(P + 20, 8, 5, 20, 0)]),          # buf[:, :5] into buf[:, 5:10]
    (-4, [(P, 8, 5, 20, 0)], [(P + 16, 8, 5, 20, 0)]),          # into buf[:, 4:9]
    (-4, [(P, 8, 5, 20, 0)], [(P, 8, 5, 21, 0)]),               # same address, another pitch
    (-4, [(P, 8, 5, 20, 0)], [(P, 8, 5, 5, 0)]),                # ... or without gaps
    (-4, [(P, 8, 5, 5, 0)], [(P, 8, 5, 20, 0)]),
    (-4, [(P, 8, 5, 20, 0)], [(P + 40, 8, 5, 5, 0)]),
    (-3, [(P, 2, 5, 20, 0)], [(P + 20, 2, 5, 5, 0)]),           # within the first gap
    (-3, [(P + 20, 2, 5, 5, 0)], [(P, 2, 5, 20, 0)]),
    (-4, [(P, 2, 5, 20, 0), (FAR, 2, 5, 20, 0)], [(FAR, 2, 5, 20, 0), (P, 2, 5, 20, 0)]),
    (-3, [(P, 2, 5, 20, 0), (FAR, 2, 5, 20, 0)], [(P, 2, 5, 20, 0), (FAR, 2, 5, 20, 0)]),
    (-3, [(P, 2, 5, 20, 0), (P + 20, 2, 5, 20, 0), (FAR, 4, 4, 4, 0)],
     [(P, 2, 5, 20, 0), (P + 20, 2, 5, 20, 0), (FAR, 4, 4, 4, 0)]),
    (-4, [(P, 2, 5, 20, 0), (P + 20, 2, 5, 20, 0)], [(P, 2, 5, 20, 0), (P + 20, 2, 5, 40, 0)]),
]


@pytest.mark.parametrize("want,a,b", PAIRS)
def test_between_sets(lib, want, a, b):
    assert _clip(lib, a, b) == want


def test_between_sets_against_enumeration(lib):
    """A random tensor of one set over its place of the other, over another's or
    beside all, against their bytes one by one."""
    rng = random.Random(4)
    seen = {-3: 0, -4: 0}
    for _ in range(4000):
        a = _random_entries(rng, 2)
        b = [(e[0] if rng.random() < 0.5 else P + rng.randrange(60) * 4, e[1], e[2],
              e[3] if rng.random() < 0.7 else e[2] + rng.randrange(6), e[4]) for e in a]
        if _fill(lib, a)[0] != 0 or _fill(lib, b)[0] != 0:
            continue
        runs = lambda e: (e[0], e[3] if e[1] > 1 else 0)  # noqa: E731
        want = -4 if any(_bytes(a[i]) & _bytes(b[j]) and not (i == j and runs(a[i]) == runs(b[j]))
                         for i in range(2) for j in range(2)) else -3
        assert _clip(lib, a, b) == want, (a, b)
        seen[want] += 1
    assert min(seen.values()) > 300, seen
