"""Calls and their streams: a gradient set's device table while calls on other
streams than its own read it (the set may be dropped as soon as the call
returns), and the handle of the current stream."""
import contextlib
import types

import pytest
import torch

import mxfp4_microscaled_precision_amd as mx_package


class _Table:
    """In the place of the device table: notes the streams it is said to be used on."""

    def __init__(self):
        self.used = []

    def record_stream(self, stream):
        self.used.append(stream)


@pytest.mark.parametrize("handle,used", [(7, ["side"]), (3, [])])
@pytest.mark.parametrize("call", ["norm", "clip", "clip out"])
def test_table_is_recorded_on_the_call_s_stream(monkeypatch, call, handle, used):
    """Sets made on stream 3, called on stream `handle` (no GPU: the library and
    the streams are stand-ins)."""
    def a_set():
        s = object.__new__(mx_package.GradSet)
        s.device, s.desc, s._home, s._table = torch.device("cuda", 0), None, 3, _Table()
        return s
    monkeypatch.setattr(mx_package, "_lib", types.SimpleNamespace(
        mx_grad_norm=lambda *a: 0, mx_grad_clip=lambda *a: 0, mx_grad_workspace=lambda: 8))
    monkeypatch.setattr(mx_package, "_place",
                        lambda device, stream: (contextlib.nullcontext(), handle))
    monkeypatch.setattr(mx_package, "_norm_buffers",
                        lambda device, lib: (torch.empty(()), torch.empty(8), 8))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "side")
    s, o = a_set(), a_set()
    if call == "norm":
        mx_package.grad_norm(s)
    elif call == "clip":
        mx_package.clip_grad_norm(s, 1.0)
    else:
        mx_package.clip_grad_norm(s, 1.0, out=o)
    assert s._table.used == used
    assert o._table.used == (used if call == "clip out" else [])


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_dropped_while_a_side_stream_runs(mx, raw):
    """The table's memory is not handed out again while a call on a side stream,
    behind other work there, still has to read it."""
    g = torch.full((1000,), 2.0, device="cuda")
    out = torch.zeros_like(g)
    big = torch.ones(1 << 28, device="cuda")                # 1 GiB, to keep the side stream busy
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sets = [mx.GradSet([t]) for t in (g, out)]
    tables = [(s.desc.table, s.desc.table_bytes) for s in sets]
    with torch.cuda.stream(side):
        for _ in range(100):
            big.mul_(1.0)
    mx.clip_grad_norm(sets[0], 1.0, out=sets[1], stream=side.cuda_stream if raw else side)
    del sets
    new = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _, n in tables * 8]
    assert not side.query(), "the side stream was done too early for this test to show anything"
    for at, n in tables:
        for t in new:
            assert t.data_ptr() + t.numel() <= at or at + n <= t.data_ptr()
    torch.cuda.synchronize()
    norm = 2.0 * 1000 ** 0.5
    # coef and the product round once each
    assert torch.all((out.double() - 2.0 / (norm + 1e-6)).abs() <= 2 * 2.0 ** -24 * 2.0 / norm)


@pytest.mark.parametrize("shortcut", [True, False])
def test_current_stream_with_and_without_torch_s_shortcut(monkeypatch, shortcut):
    """The handle of the current stream comes from a private function of torch,
    or from the public one where that is gone (stand-ins, no GPU)."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=9))
    if shortcut:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 8, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    place, handle = mx_package._place(torch.device("cuda", 0), None)
    assert handle == (8 if shortcut else 9)
    with place:
        pass
