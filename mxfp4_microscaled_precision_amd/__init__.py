"""MXFP4 linear layers on MI355X (gfx950): Python binding of libmxfp4.so.

The binding only marshals arguments: PyTorch provides device memory and the
current HIP stream, and every step of the computation runs in the library's
HIP kernels. There is no CPU fallback; if the library is missing, loading it
raises.

    q_x = quantize(x_bf16, axis=1, rotate="hadamard", round="rne", seed=0)
    q_w = quantize(w_bf16, axis=1, rotate="hadamard", seed=1 << 32)
    y = linear("fprop", q_x, q_w, out_dtype="bf16")

The three GEMMs and their operand axes (36Kr article "Neue Studie von AMD
durchbricht die bestehende Erkenntnis ...", section "Fehlerdiagnoseexperiment"):
    fprop: A = X  [T, in]  axis 1, B = W [out, in] axis 1 -> Y  [T, out]
    dgrad: A = dY [T, out] axis 1, B = W [out, in] axis 0 -> dX [T, in]
    wgrad: A = dY [T, out] axis 0, B = X [T, in]   axis 0 -> dW [out, in]

Around the linears of a training step: rmsnorm_quantize writes the packed
operands of the normalised residual stream, rmsnorm_backward is its gradient,
and clip_grad_norm scales the gradients by their global norm. linear_fused
computes a linear with its bias, activation, gate and residual in one launch,
linear_act_backward the gradient through the activation, linear_grouped the
linears of all experts over rows that quantize_grouped gathered.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple, Optional, Tuple

__all__ = [
    "LIB_PATH", "MxError", "QTensorDesc", "QTensor", "load_library", "library_symbols",
    "status_string", "version", "last_hip_error", "quantize_sizes", "quantize", "quantize_dual",
    "quantize_pair",
    "quantize_fp8_sizes", "quantize_fp8", "linear", "linear_batched", "dequantize",
    "NormDesc", "NormGradDesc", "GradDesc", "GradSetDesc", "RMSNormQuantized",
    "rmsnorm_quantize", "rmsnorm_backward", "GradSet", "grad_norm", "clip_grad_norm",
    "EpilogueDesc", "GroupedDesc", "GroupedSourceDesc", "GroupedQuantized", "packed_operand",
    "quantize_grouped_sizes", "quantize_grouped", "linear_fused", "linear_act_backward",
    "linear_grouped",
    "ROTATE", "ROUND", "FORMATS", "OPS", "OUT_DTYPES", "OP_AXES", "ACTIVATIONS", "AXIS_GROUPED",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4.so")

ROTATE = {"none": 0, "hadamard": 1, "rand_sign_hadamard": 2, "hadamard16": 3}
ROUND = {"rne": 0, "sr": 1}
FORMATS = {"fp4_e2m1": 0, "fp8_e4m3": 1}
OPS = {"fprop": 0, "dgrad": 1, "wgrad": 2}
OUT_DTYPES = {"f32": 0, "bf16": 1}
# (A axis, B axis) each op needs
OP_AXES = {"fprop": (1, 1), "dgrad": (1, 0), "wgrad": (0, 0)}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
# the axis of a grouped operand whose blocks run along its rows, group by group
AXIS_GROUPED = 2

MX_OK = 0


class MxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {status_string(status)} ({status})"
        if status == -7:
            msg += f" [{load_library().mx_last_hip_error().decode()}]"
        super().__init__(msg)


class QTensorDesc(ctypes.Structure):
    """Mirror of struct mx_qtensor in include/mxfp4.h."""
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("axis", ctypes.c_int32),
        ("block", ctypes.c_int32),
        ("rotate", ctypes.c_int32),
        ("round", ctypes.c_int32),
        ("seed", ctypes.c_uint64),
        ("format", ctypes.c_int32),
    ]


class NormDesc(ctypes.Structure):
    """Mirror of struct mx_norm in include/mxfp4.h."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("residual", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("h", ctypes.c_void_p),
        ("rstd", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ldx", ctypes.c_int64),
        ("ldr", ctypes.c_int64),
        ("ldh", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
        ("eps", ctypes.c_double),
    ]


class NormGradDesc(ctypes.Structure):
    """Mirror of struct mx_norm_grad in include/mxfp4.h."""
    _fields_ = [
        ("dy", ctypes.c_void_p),
        ("h", ctypes.c_void_p),
        ("dres", ctypes.c_void_p),
        ("rstd", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("dh", ctypes.c_void_p),
        ("dweight", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("lddy", ctypes.c_int64),
        ("ldh", ctypes.c_int64),
        ("ldres", ctypes.c_int64),
        ("lddh", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("weight_dtype", ctypes.c_int32),
    ]


class GradDesc(ctypes.Structure):
    """Mirror of struct mx_grad in include/mxfp4.h."""
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
    ]


class GradSetDesc(ctypes.Structure):
    """Mirror of struct mx_grad_set in include/mxfp4.h."""
    _fields_ = [
        ("grads", ctypes.POINTER(GradDesc)),
        ("count", ctypes.c_int32),
        ("host_table", ctypes.c_void_p),
        ("table", ctypes.c_void_p),
        ("table_bytes", ctypes.c_size_t),
        ("chunks", ctypes.c_int64),
        ("chunk", ctypes.c_int64),
    ]


class EpilogueDesc(ctypes.Structure):
    """Mirror of struct mx_epilogue in include/mxfp4.h."""
    _fields_ = [
        ("activation", ctypes.c_int32),
        ("gradient", ctypes.c_int32),
        ("bias", ctypes.c_void_p),
        ("bias_dtype", ctypes.c_int32),
        ("mul", ctypes.c_void_p),
        ("residual", ctypes.c_void_p),
        ("pre", ctypes.c_void_p),
        ("dmul", ctypes.c_void_p),
        ("ldmul", ctypes.c_int64),
        ("ldres", ctypes.c_int64),
        ("ldpre", ctypes.c_int64),
        ("lddmul", ctypes.c_int64),
    ]


class GroupedDesc(ctypes.Structure):
    """Mirror of struct mx_grouped in include/mxfp4.h."""
    _fields_ = [
        ("q", QTensorDesc),
        ("groups", ctypes.c_int32),
        ("group_rows", ctypes.c_int64),
    ]


class GroupedSourceDesc(ctypes.Structure):
    """Mirror of struct mx_grouped_source in include/mxfp4.h."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("src_rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("index", ctypes.c_void_p),
        ("index_bits", ctypes.c_int32),
        ("rows", ctypes.c_int64),
        ("groups", ctypes.c_int32),
        ("group_rows", ctypes.c_int64),
        ("ends", ctypes.c_void_p),
    ]


_lib: Optional[ctypes.CDLL] = None

_SIGNATURES = {
    "mx_quantize_sizes": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                         ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t),
                                         ctypes.POINTER(ctypes.c_size_t)]),
    "mx_quantize_fp8_sizes": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t),
                                             ctypes.POINTER(ctypes.c_size_t)]),
    "mx_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                   ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                   ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64,
                                   ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.POINTER(QTensorDesc), ctypes.c_void_p]),
    "mx_quantize_dual": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.POINTER(QTensorDesc),
                                        ctypes.POINTER(QTensorDesc), ctypes.c_void_p]),
    "mx_quantize_pair": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.POINTER(QTensorDesc),
                                        ctypes.POINTER(QTensorDesc), ctypes.c_void_p]),
    "mx_quantize_fp8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_int32, ctypes.c_uint64, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.POINTER(QTensorDesc),
                                       ctypes.c_void_p]),
    "mx_linear": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(QTensorDesc),
                                 ctypes.POINTER(QTensorDesc), ctypes.c_void_p, ctypes.c_int64,
                                 ctypes.c_int32, ctypes.c_void_p]),
    "mx_linear_batched": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32,
                                         ctypes.POINTER(QTensorDesc), ctypes.POINTER(QTensorDesc),
                                         ctypes.POINTER(ctypes.c_void_p), ctypes.c_int64,
                                         ctypes.c_int32, ctypes.c_void_p]),
    "mx_dequantize": (ctypes.c_int, [ctypes.POINTER(QTensorDesc), ctypes.c_void_p,
                                     ctypes.c_int64, ctypes.c_void_p]),
    "mx_rmsnorm_quantize": (ctypes.c_int, [ctypes.POINTER(NormDesc), ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_uint64, ctypes.c_uint64, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.POINTER(QTensorDesc),
                                           ctypes.POINTER(QTensorDesc), ctypes.c_void_p]),
    "mx_rmsnorm_backward_workspace": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64,
                                                     ctypes.POINTER(ctypes.c_size_t)]),
    "mx_rmsnorm_backward": (ctypes.c_int, [ctypes.POINTER(NormGradDesc), ctypes.c_void_p,
                                           ctypes.c_size_t, ctypes.c_void_p]),
    "mx_grad_set_size": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(GradDesc),
                                        ctypes.POINTER(ctypes.c_size_t)]),
    "mx_grad_set_fill": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(GradDesc),
                                        ctypes.c_void_p, ctypes.c_size_t,
                                        ctypes.POINTER(GradSetDesc)]),
    "mx_grad_workspace": (ctypes.c_size_t, []),
    "mx_grad_norm": (ctypes.c_int, [ctypes.POINTER(GradSetDesc), ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "mx_grad_clip": (ctypes.c_int, [ctypes.POINTER(GradSetDesc), ctypes.POINTER(GradSetDesc),
                                    ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]),
    "mx_linear_fused": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(QTensorDesc),
                                       ctypes.POINTER(QTensorDesc),
                                       ctypes.POINTER(EpilogueDesc), ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p]),
    "mx_quantize_grouped_sizes": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                                 ctypes.c_int64, ctypes.c_int32,
                                                 ctypes.POINTER(ctypes.c_size_t),
                                                 ctypes.POINTER(ctypes.c_size_t)]),
    "mx_quantize_grouped_workspace": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int64,
                                                     ctypes.c_int32, ctypes.c_int64,
                                                     ctypes.POINTER(ctypes.c_size_t)]),
    "mx_quantize_grouped": (ctypes.c_int, [ctypes.POINTER(GroupedSourceDesc), ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_int32, ctypes.c_uint64,
                                           ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_size_t,
                                           ctypes.POINTER(GroupedDesc),
                                           ctypes.POINTER(GroupedDesc), ctypes.c_void_p]),
    "mx_linear_grouped": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(GroupedDesc),
                                         ctypes.POINTER(GroupedDesc), ctypes.c_void_p,
                                         ctypes.POINTER(EpilogueDesc), ctypes.c_void_p,
                                         ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p]),
    "mx_status_string": (ctypes.c_char_p, [ctypes.c_int32]),
    "mx_version": (ctypes.c_char_p, []),
    "mx_last_hip_error": (ctypes.c_char_p, []),
}


def library_symbols() -> Tuple[str, ...]:
    return tuple(_SIGNATURES)


def _hip_runtimes_mapped():
    try:
        with open("/proc/self/maps") as fh:
            return sorted({ln.split()[-1] for ln in fh if "libamdhip64" in ln})
    except OSError:
        return []


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmxfp4.so (built by mxfp4_microscaled_precision_amd.build).

    torch is imported first: PyTorch-ROCm ships its own HIP runtime under the
    same soname, and the library must bind to that one so that torch's streams
    and allocations are valid for its launches. Two HIP runtimes in one process
    is refused with an error.
    """
    global _lib
    if _lib is not None and path is None:
        return _lib
    import torch  # noqa: F401  (binds libamdhip64 to torch's runtime first)
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it with `python -m mxfp4_microscaled_precision_amd.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(p)
    runtimes = _hip_runtimes_mapped()
    if len(runtimes) > 1:
        raise RuntimeError("two HIP runtimes are loaded in this process (%s); load torch "
                           "before libmxfp4.so" % ", ".join(runtimes))
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().mx_status_string(int(status)).decode()


def version() -> str:
    return load_library().mx_version().decode()


def last_hip_error() -> str:
    return load_library().mx_last_hip_error().decode()


def _check(status: int, where: str) -> None:
    if status != MX_OK:
        raise MxError(status, where)


def quantize_sizes(rows: int, cols: int, axis: int, block: int = 32) -> Tuple[int, int]:
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().mx_quantize_sizes(rows, cols, axis, block, ctypes.byref(cb),
                                            ctypes.byref(sb)), "mx_quantize_sizes")
    return cb.value, sb.value


def quantize_fp8_sizes(rows: int, cols: int, axis: int, block: int = 32) -> Tuple[int, int]:
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().mx_quantize_fp8_sizes(rows, cols, axis, block, ctypes.byref(cb),
                                                ctypes.byref(sb)), "mx_quantize_fp8_sizes")
    return cb.value, sb.value


def _stream_handle(device, stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


class QTensor:
    """A quantized operand: flat uint8 buffers holding the tiled codes and
    scales (layout in include/mxfp4.h, struct mx_qtensor) plus the C
    descriptor that points at them. Where its source's rows belong to groups:
    how many, and the rows of each, or -1 where the ends tell (struct
    mx_grouped)."""

    def __init__(self, codes, scales, desc: QTensorDesc, groups: Optional[int] = None,
                 group_rows: int = -1):
        self.codes = codes
        self.scales = scales
        self.desc = desc
        self.groups = groups
        self.group_rows = group_rows

    @property
    def axis(self) -> int:
        return self.desc.axis

    @property
    def source_shape(self) -> Tuple[int, int]:
        return (self.desc.rows, self.desc.cols)

    @property
    def format(self) -> str:
        return {v: k for k, v in FORMATS.items()}[self.desc.format]

    @property
    def mn(self) -> int:
        return self.desc.rows if self.desc.axis == 1 else self.desc.cols

    @property
    def k(self) -> int:
        return self.desc.cols if self.desc.axis == 1 else self.desc.rows


def _source_extents(x) -> Tuple[int, int, int]:
    """(rows, cols, ld) of a 2-D bf16 CUDA source; raises for anything else."""
    import torch
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA (HIP) tensor; there is no CPU path")
    if x.numel() > 0 and x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else max(cols, 8 * ((cols + 7) // 8))
    return rows, cols, ld


def quantize(x, axis: int, rotate: str = "hadamard", round: str = "rne", seed: int = 0,
             codes=None, scales=None, stream=None) -> QTensor:
    """Rotate + quantize a 2-D bf16 CUDA tensor along `axis` (see mx_quantize).

    x may be a row-strided view (stride(1) == 1). codes / scales may be
    preallocated uint8 tensors of at least the sizes quantize_sizes returns.
    """
    import torch
    lib = load_library()
    rows, cols, ld = _source_extents(x)
    cb, sb = quantize_sizes(rows, cols, axis)
    if codes is None:
        codes = torch.empty((cb,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((sb,), dtype=torch.uint8, device=x.device)
    if codes.numel() < cb or scales.numel() < sb:
        raise ValueError("codes / scales buffers too small")
    desc = QTensorDesc()
    st = lib.mx_quantize(x.data_ptr() if x.numel() else None, rows, cols, ld, axis, 32,
                         ROTATE[rotate], ROUND[round], seed & 0xFFFFFFFFFFFFFFFF,
                         codes.data_ptr() if codes.numel() else None,
                         scales.data_ptr() if scales.numel() else None,
                         ctypes.byref(desc), _stream_handle(x.device, stream))
    _check(st, "mx_quantize")
    return QTensor(codes, scales, desc)


def quantize_pair(xa, xb, rotate: str = "hadamard", round: str = "rne", seed_a: int = 0,
                  seed_b: int = 0, stream=None) -> Tuple[QTensor, QTensor]:
    """Axis-1 quantizations of two 2-D bf16 CUDA tensors with the same column
    count in one launch (see mx_quantize_pair): returns (A operand, B operand),
    byte-identical to quantize(xa, 1, ...) and quantize(xb, 1, ...)."""
    import torch
    lib = load_library()
    ra, cols, lda = _source_extents(xa)
    rb, cols_b, ldb = _source_extents(xb)
    if cols != cols_b:
        raise ValueError("quantize_pair needs sources with the same column count")
    out = []
    for rows in (ra, rb):
        cb, sb = quantize_sizes(rows, cols, 1)
        out.append((torch.empty((cb,), dtype=torch.uint8, device=xa.device),
                    torch.empty((sb,), dtype=torch.uint8, device=xa.device)))
    (ca, sa), (cb_, sb_) = out
    da, db = QTensorDesc(), QTensorDesc()
    ptr = lambda t: t.data_ptr() if t.numel() else None  # noqa: E731
    st = lib.mx_quantize_pair(ptr(xa), ra, lda, ptr(xb), rb, ldb, cols, 32, ROTATE[rotate],
                              ROUND[round], seed_a & 0xFFFFFFFFFFFFFFFF,
                              seed_b & 0xFFFFFFFFFFFFFFFF, ptr(ca), ptr(sa), ptr(cb_), ptr(sb_),
                              ctypes.byref(da), ctypes.byref(db), _stream_handle(xa.device, stream))
    _check(st, "mx_quantize_pair")
    return QTensor(ca, sa, da), QTensor(cb_, sb_, db)


def quantize_dual(x, rotate: str = "hadamard", round: str = "rne", seed1: int = 0,
                  seed0: int = 0, stream=None) -> Tuple[QTensor, QTensor]:
    """Both orientations of a 2-D bf16 CUDA tensor from one read of it (see
    mx_quantize_dual): returns (axis-1 operand, axis-0 operand)."""
    import torch
    lib = load_library()
    rows, cols, ld = _source_extents(x)
    out = []
    for axis in (1, 0):
        cb, sb = quantize_sizes(rows, cols, axis)
        out.append((torch.empty((cb,), dtype=torch.uint8, device=x.device),
                    torch.empty((sb,), dtype=torch.uint8, device=x.device)))
    (c1, s1), (c0, s0) = out
    d1, d0 = QTensorDesc(), QTensorDesc()
    ptr = lambda t: t.data_ptr() if t.numel() else None  # noqa: E731
    st = lib.mx_quantize_dual(ptr(x), rows, cols, ld, 32, ROTATE[rotate], ROUND[round],
                              seed1 & 0xFFFFFFFFFFFFFFFF, seed0 & 0xFFFFFFFFFFFFFFFF,
                              ptr(c1), ptr(s1), ptr(c0), ptr(s0), ctypes.byref(d1),
                              ctypes.byref(d0), _stream_handle(x.device, stream))
    _check(st, "mx_quantize_dual")
    return QTensor(c1, s1, d1), QTensor(c0, s0, d0)


def quantize_fp8(x, axis: int, rotate: str = "hadamard", seed: int = 0, codes=None,
                 scales=None, stream=None) -> QTensor:
    """Rotate + quantize into MXFP8 with E4M3 elements, the FP8 comparator
    (see mx_quantize_fp8; nearest rounding only). Arguments as for quantize."""
    import torch
    lib = load_library()
    rows, cols, ld = _source_extents(x)
    cb, sb = quantize_fp8_sizes(rows, cols, axis)
    if codes is None:
        codes = torch.empty((cb,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((sb,), dtype=torch.uint8, device=x.device)
    if codes.numel() < cb or scales.numel() < sb:
        raise ValueError("codes / scales buffers too small")
    desc = QTensorDesc()
    st = lib.mx_quantize_fp8(x.data_ptr() if x.numel() else None, rows, cols, ld, axis, 32,
                             ROTATE[rotate], seed & 0xFFFFFFFFFFFFFFFF,
                             codes.data_ptr() if codes.numel() else None,
                             scales.data_ptr() if scales.numel() else None,
                             ctypes.byref(desc), _stream_handle(x.device, stream))
    _check(st, "mx_quantize_fp8")
    return QTensor(codes, scales, desc)


def linear(op: str, A: QTensor, B: QTensor, out_dtype: str = "f32", out=None,
           stream=None):
    """One GEMM of the triple (see mx_linear); returns C [M, N] (fp32 or bf16).
    Two MXFP8 operands (quantize_fp8) run the E4M3 comparator GEMM."""
    import torch
    lib = load_library()
    M, N = A.mn, B.mn
    dt = torch.float32 if out_dtype == "f32" else torch.bfloat16
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=A.codes.device)
    if out.dtype != dt or out.dim() != 2 or tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong dtype or shape")
    if out.numel() and out.stride(1) != 1:
        raise ValueError("out must have unit column stride")
    ldc = out.stride(0) if M > 1 else max(N, 4)
    st = lib.mx_linear(OPS[op], ctypes.byref(A.desc), ctypes.byref(B.desc),
                       out.data_ptr() if out.numel() else None, ldc, OUT_DTYPES[out_dtype],
                       _stream_handle(A.codes.device, stream))
    _check(st, "mx_linear")
    return out


def linear_batched(op: str, As, Bs, out_dtype: str = "f32", outs=None, stream=None):
    """Several GEMMs of one op and one shape in one launch (see
    mx_linear_batched): C[i] = linear(op, As[i], Bs[i]); returns the list of
    C [M, N] (fp32 or bf16), bitwise identical to separate linear calls."""
    import torch
    lib = load_library()
    n = len(As)
    if len(Bs) != n:
        raise ValueError("As and Bs differ in length")
    M, N = As[0].mn, Bs[0].mn
    dt = torch.float32 if out_dtype == "f32" else torch.bfloat16
    if outs is None:
        outs = [torch.empty((M, N), dtype=dt, device=As[0].codes.device) for _ in range(n)]
    if len(outs) != n:
        raise ValueError("outs differs in length")
    lds = set()
    for o in outs:
        if o.dtype != dt or o.dim() != 2 or tuple(o.shape) != (M, N):
            raise ValueError("an output has the wrong dtype or shape")
        if o.numel() and o.stride(1) != 1:
            raise ValueError("outputs must have unit column stride")
        lds.add(o.stride(0) if M > 1 else max(N, 4))
    if len(lds) != 1:
        raise ValueError("outputs must share one leading dimension")
    da = (QTensorDesc * n)(*[q.desc for q in As])
    db = (QTensorDesc * n)(*[q.desc for q in Bs])
    cs = (ctypes.c_void_p * n)(*[o.data_ptr() if o.numel() else None for o in outs])
    st = lib.mx_linear_batched(OPS[op], n, da, db, cs, lds.pop(), OUT_DTYPES[out_dtype],
                               _stream_handle(As[0].codes.device, stream))
    _check(st, "mx_linear_batched")
    return outs


def dequantize(q: QTensor, out=None, stream=None):
    """fp32 values of a quantized operand in its source's shape [rows, cols]
    (see mx_dequantize): sign * E2M1 (or E4M3) value * 2^(scale - 127)."""
    import torch
    lib = load_library()
    rows, cols = q.source_shape
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=q.codes.device)
    if out.dtype != torch.float32 or out.dim() != 2 or tuple(out.shape) != (rows, cols):
        raise ValueError("out must be a float32 tensor of the source's shape")
    if out.numel() and out.stride(1) != 1:
        raise ValueError("out must have unit column stride")
    ld = out.stride(0) if rows > 1 else max(cols, 1)
    st = lib.mx_dequantize(ctypes.byref(q.desc), out.data_ptr() if out.numel() else None, ld,
                           _stream_handle(q.codes.device, stream))
    _check(st, "mx_dequantize")
    return out


_HERE = contextlib.nullcontext()


def _place(device, stream):
    """(context, stream handle) of a call on `device`: inside the context the
    device is current and torch allocates for the stream that the call runs on,
    so that neither an output nor a workspace is memory another stream may
    still be using."""
    import torch
    if stream is None:
        # current_stream without its stream object, where torch still has that
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        handle = raw(device.index) if raw else torch.cuda.current_stream(device).cuda_stream
        here = device.index == torch.cuda.current_device()
        return (_HERE if here else torch.cuda.device(device)), handle
    if not hasattr(stream, "cuda_stream"):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    if stream.device != device:
        raise ValueError("stream is on another device than the tensors")
    return torch.cuda.stream(stream), stream.cuda_stream


_ROW_DTYPES = {}


def _row_dtype(t, name: str) -> int:
    if not _ROW_DTYPES:
        import torch
        _ROW_DTYPES.update({torch.float32: OUT_DTYPES["f32"], torch.bfloat16: OUT_DTYPES["bf16"]})
    dtype = _ROW_DTYPES.get(t.dtype)
    if dtype is None:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return dtype


def _first_rows(t, name: str) -> Tuple[int, int]:
    """(rows, cols) of the 2-D CUDA matrix that sets a call's type and shape."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor; there is no CPU path")
    return shape


def _rows_of(t, name: str, rows: int, cols: int, dtype, device) -> Tuple[Optional[int], int]:
    """(address, leading dimension) of a matrix of the given shape, type and
    device with unit column stride."""
    shape = t.shape
    if (len(shape) != 2 or shape[0] != rows or shape[1] != cols or t.dtype is not dtype
            or t.device != device):
        raise ValueError(f"{name} must have the type, shape and device of the other rows")
    if rows == 0 or cols == 0:
        return None, (cols + 7) // 8 * 8
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), ld if rows > 1 else (cols + 7) // 8 * 8


def _vector(t, name: str, n: int, device):
    shape = t.shape
    if len(shape) != 1 or shape[0] != n or t.device != device:
        raise ValueError(f"{name} must be a 1-D tensor of {n} elements on the rows' device")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() if n else None


@functools.lru_cache(maxsize=256)
def _norm_sizes(fmt: int, rows: int, cols: int, dual: bool) -> Tuple[int, ...]:
    """Bytes of codes1, scales1 (and codes0, scales0), a function of the shape."""
    sizes = quantize_fp8_sizes if fmt else quantize_sizes
    return sizes(rows, cols, 1) + (sizes(rows, cols, 0) if dual else ())


@functools.lru_cache(maxsize=256)
def _backward_workspace(rows: int, cols: int) -> int:
    need = ctypes.c_size_t()
    _check(load_library().mx_rmsnorm_backward_workspace(rows, cols, need),
           "mx_rmsnorm_backward_workspace")
    return need.value


class RMSNormQuantized(NamedTuple):
    """What rmsnorm_quantize returns: the axis-1 and axis-0 operands of y (q0 is
    None without dual), the residual stream h and rstd per row."""
    q1: QTensor
    q0: Optional[QTensor]
    h: object
    rstd: object


def rmsnorm_quantize(x, weight, residual=None, eps: float = 1e-5, format: str = "fp4_e2m1",
                     dual: bool = False, rotate: str = "hadamard", round: str = "rne",
                     seed1: int = 0, seed0: int = 0, h=None, stream=None) -> RMSNormQuantized:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, and y rotated
    and quantized into the operands the linears read (see mx_rmsnorm_quantize).

    x, residual: 2-D bf16 or fp32 CUDA tensors (row-strided views allowed);
    weight: bf16 or fp32 [cols]. format, rotate, round and the seeds are those
    of quantize_dual / quantize_fp8; dual adds the axis-0 operand. h: where the
    stream is written, may be residual or x itself to update it in place; x is
    returned as h where there is no residual. stream: a torch stream or a raw
    handle to run on instead of the current one; the outputs are allocated for
    it, and the inputs must be ready there.
    """
    import torch
    lib = _lib or load_library()
    rows, cols = _first_rows(x, "x")
    kind, dtype, device = x.dtype, _row_dtype(x, "x"), x.device
    xp, ldx = _rows_of(x, "x", rows, cols, kind, device)
    wp = _vector(weight, "weight", cols, device)
    rp, ldr = ((None, 0) if residual is None
               else _rows_of(residual, "residual", rows, cols, kind, device))
    fmt = FORMATS[format]
    size = _norm_sizes(fmt, rows, cols, bool(dual))
    place, handle = _place(device, stream)
    with place:
        if residual is None:
            if h is not None and h is not x:
                raise ValueError("without a residual h is x itself")
            h, hp, ldh = x, None, 0
        elif h is None:
            h = (torch.empty_like(x) if ldx == cols and rows > 1
                 else torch.empty((rows, cols), dtype=kind, device=device))
            hp, ldh = h.data_ptr(), cols
        else:
            hp, ldh = _rows_of(h, "h", rows, cols, kind, device)
        rstd = torch.empty(rows, dtype=torch.float32, device=device)
        buf = [torch.empty(b, dtype=torch.uint8, device=device) for b in size]
        ptr = [b.data_ptr() or None for b in buf] + [None, None]
        n = NormDesc(xp, rp, wp, hp, rstd.data_ptr() or None, rows, cols, ldx, ldr, ldh, dtype,
                     _row_dtype(weight, "weight"), eps)
        d1, d0 = QTensorDesc(), QTensorDesc()
        st = lib.mx_rmsnorm_quantize(n, fmt, 32, ROTATE[rotate], ROUND[round],
                                     seed1 & 0xFFFFFFFFFFFFFFFF, seed0 & 0xFFFFFFFFFFFFFFFF,
                                     ptr[0], ptr[1], ptr[2], ptr[3], d1, d0, handle)
    _check(st, "mx_rmsnorm_quantize")
    if not dual:
        return RMSNormQuantized(QTensor(buf[0], buf[1], d1), None, h, rstd)
    if not (rows and cols):     # empty operands have no buffers to tell the call by
        d0 = QTensorDesc(None, None, rows, cols, 0, 32, ROTATE[rotate], ROUND[round],
                         seed0 & 0xFFFFFFFFFFFFFFFF, fmt)
    return RMSNormQuantized(QTensor(buf[0], buf[1], d1), QTensor(buf[2], buf[3], d0), h, rstd)


def rmsnorm_backward(dy, h, rstd, weight, dres=None, dh=None, stream=None):
    """Gradient of rmsnorm_quantize (see mx_rmsnorm_backward): returns (dh,
    dweight). dy: gradient of y; h, rstd: what the forward call returned; dres:
    the gradient that reaches h past the norm. dh is the gradient of x and of
    residual; it may be written over dy or dres. dweight is fp32."""
    import torch
    lib = _lib or load_library()
    rows, cols = _first_rows(dy, "dy")
    kind, dtype, device = dy.dtype, _row_dtype(dy, "dy"), dy.device
    yp, lddy = _rows_of(dy, "dy", rows, cols, kind, device)
    hp, ldh = _rows_of(h, "h", rows, cols, kind, device)
    rp, ldres = (None, 0) if dres is None else _rows_of(dres, "dres", rows, cols, kind, device)
    if rstd.dtype is not torch.float32:
        raise ValueError("rstd must be float32")
    sp = _vector(rstd, "rstd", rows, device)
    wp = _vector(weight, "weight", cols, device)
    need = _backward_workspace(rows, cols)
    place, handle = _place(device, stream)
    with place:
        if dh is None:
            dh = (torch.empty_like(dy) if lddy == cols and rows > 1
                  else torch.empty((rows, cols), dtype=kind, device=device))
            dp, lddh = dh.data_ptr() or None, cols
        else:
            dp, lddh = _rows_of(dh, "dh", rows, cols, kind, device)
        dweight = torch.empty(cols, dtype=torch.float32, device=device)
        work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        g = NormGradDesc(yp, hp, rp, sp, wp, dp, dweight.data_ptr() or None, rows, cols, lddy, ldh,
                         ldres, lddh, dtype, _row_dtype(weight, "weight"))
        st = lib.mx_rmsnorm_backward(g, work.data_ptr() if need else None, need, handle)
    _check(st, "mx_rmsnorm_backward")
    return dh, dweight


class GradSet:
    """Gradient tensors laid out once for grad_norm and clip_grad_norm (see
    mx_grad_set): fp32 and bf16 CUDA tensors of one device, mixed as they come,
    contiguous or (1-D and 2-D) row-strided, no element in two of them. It holds the tensors and their
    addresses: make another when one is replaced. It cannot be made while a
    graph is captured (its table is copied to the device), and a captured graph
    that uses it needs it for as long as the graph is replayed. It may be dropped
    while a call on any stream still runs; a raw handle's stream has to live as
    long as the set."""

    def __init__(self, tensors):
        import torch
        lib = load_library()
        self.tensors = list(tensors)
        self.device = self.tensors[0].device if self.tensors else None
        self._grads = (GradDesc * max(1, len(self.tensors)))()
        for g, t in zip(self._grads, self.tensors):
            if not t.is_cuda or t.device != self.device:
                raise ValueError("gradients must be CUDA (HIP) tensors of one device")
            g.dtype = _row_dtype(t, "a gradient")
            g.data = t.data_ptr() if t.numel() else None
            if t.dim() == 1:
                g.rows, g.cols, g.ld = t.shape[0], 1, t.stride(0)
            elif t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1):
                g.rows, g.cols, g.ld = t.shape[0], t.shape[1], t.stride(0)
            elif t.is_contiguous():
                g.rows, g.cols, g.ld = 1, t.numel(), t.numel()
            else:
                raise ValueError("a gradient must be contiguous or a row-strided matrix")
        need = ctypes.c_size_t()
        _check(lib.mx_grad_set_size(len(self.tensors), self._grads, ctypes.byref(need)),
               "mx_grad_set_size")
        self._host = torch.zeros((need.value,), dtype=torch.uint8)
        self.desc = GradSetDesc()
        _check(lib.mx_grad_set_fill(len(self.tensors), self._grads,
                                    self._host.data_ptr() if need.value else None, need.value,
                                    ctypes.byref(self.desc)), "mx_grad_set_fill")
        self._table, self._home = None, 0
        if need.value:
            self._home = torch.cuda.current_stream(self.device).cuda_stream
            self._table = self._host.to(self.device)
            self.desc.table = self._table.data_ptr()

    def _used_on(self, handle: int) -> None:
        """A call on the current stream, `handle`, reads the table: where that is
        not the stream it was allocated for, its memory must not go to the next
        allocation there, should the set be dropped, before this call is done."""
        if handle != self._home and self._table is not None:
            import torch
            self._table.record_stream(torch.cuda.current_stream(self.device))


def _grads_and_device(grads):
    """A GradSet or a list of tensors as it is, and the device it is on."""
    import torch
    if not isinstance(grads, GradSet):
        grads = list(grads)
        device = grads[0].device if grads else None
    else:
        device = grads.device
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    elif device.type != "cuda":
        raise ValueError("gradients must be CUDA (HIP) tensors; there is no CPU path")
    return grads, device


def _as_set(grads) -> GradSet:
    return grads if isinstance(grads, GradSet) else GradSet(grads)


def _norm_buffers(device, lib):
    import torch
    size = lib.mx_grad_workspace()
    return (torch.empty((), dtype=torch.float32, device=device),
            torch.empty(size, dtype=torch.uint8, device=device), size)


def grad_norm(grads, stream=None):
    """Global 2-norm of a GradSet or of a list of gradients (see mx_grad_norm),
    a 0-dimensional fp32 CUDA tensor; with a GradSet nothing waits for the GPU."""
    lib = _lib or load_library()
    grads, device = _grads_and_device(grads)
    place, handle = _place(device, stream)
    with place:
        s = _as_set(grads)
        s._used_on(handle)
        norm, work, size = _norm_buffers(device, lib)
        st = lib.mx_grad_norm(s.desc, norm.data_ptr(), work.data_ptr(), size, handle)
    _check(st, "mx_grad_norm")
    return norm


def clip_grad_norm(grads, max_norm: float, out=None, stream=None):
    """Scale gradients by min(1, max_norm / (norm + 1e-6)), norm their global
    2-norm, which is returned as grad_norm returns it (see mx_grad_clip). In
    place, or into `out`: tensors of the same shapes and types. Both may be
    GradSets, made once, or lists."""
    lib = _lib or load_library()
    grads, device = _grads_and_device(grads)
    if out is not None:
        out, there = _grads_and_device(out)
        if there != device:
            raise ValueError("out must be on the gradients' device")
    place, handle = _place(device, stream)
    with place:
        s = _as_set(grads)
        o = s if out is None else _as_set(out)
        s._used_on(handle)
        if o is not s:
            o._used_on(handle)
        norm, work, size = _norm_buffers(device, lib)
        st = lib.mx_grad_clip(s.desc, o.desc, max_norm,
                              norm.data_ptr(), work.data_ptr(), size, handle)
    _check(st, "mx_grad_clip")
    return norm


@functools.lru_cache(maxsize=256)
def quantize_grouped_sizes(rows: int, cols: int, groups: int, group_rows: int = -1,
                           axis: int = AXIS_GROUPED) -> Tuple[int, int]:
    """Bytes of (codes, scales) of an operand of grouped rows: axis 1, or
    AXIS_GROUPED (see mx_quantize_grouped_sizes)."""
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().mx_quantize_grouped_sizes(rows, cols, groups, group_rows, axis, cb, sb),
           "mx_quantize_grouped_sizes")
    return cb.value, sb.value


@functools.lru_cache(maxsize=256)
def _grouped_workspace(rows: int, cols: int, groups: int, group_rows: int) -> int:
    need = ctypes.c_size_t()
    _check(load_library().mx_quantize_grouped_workspace(rows, cols, groups, group_rows, need),
           "mx_quantize_grouped_workspace")
    return need.value


def packed_operand(codes, scales, rows: int, cols: int, axis: int, rotate: str = "hadamard",
                   round: str = "rne", seed: int = 0, format: str = "fp4_e2m1",
                   groups: Optional[int] = None, group_rows: int = -1) -> QTensor:
    """The operand in existing buffers, as the quantizers laid them out (copied,
    stored and loaded again, received from another process). rows, cols, axis
    and the rest are those it was quantized with; with groups, axis 0 is the
    grouped operand of quantize_grouped."""
    import torch
    if groups is None:
        sizes = quantize_fp8_sizes if FORMATS[format] else quantize_sizes
        cb, sb = sizes(rows, cols, axis)
    else:
        if FORMATS[format]:
            raise ValueError("operands of grouped rows are MXFP4")
        if axis not in (0, 1):
            raise ValueError("axis must be 0 or 1")
        axis = axis or AXIS_GROUPED
        cb, sb = quantize_grouped_sizes(rows, cols, groups, group_rows, axis)
    for t, need in ((codes, cb), (scales, sb)):
        if t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() < need:
            raise ValueError("codes / scales must be contiguous uint8 buffers of the operand's size")
        if not t.is_cuda or t.device != codes.device:
            raise ValueError("codes and scales must be CUDA (HIP) tensors of one device")
    desc = QTensorDesc(codes.data_ptr() if cb else None, scales.data_ptr() if sb else None, rows,
                       cols, axis, 32, ROTATE[rotate], ROUND[round], seed & 0xFFFFFFFFFFFFFFFF,
                       FORMATS[format])
    return QTensor(codes, scales, desc, groups, group_rows)


class GroupedQuantized(NamedTuple):
    """What quantize_grouped returns: the axis-1 operand of the rows, the grouped
    axis-0 operand (None without dual) and the groups' column sums (None unless
    asked for)."""
    q1: QTensor
    q0: Optional[QTensor]
    sums: object


def _ends(ends, groups: Optional[int], device):
    """(address, groups) of the groups' ends."""
    import torch
    if ends.dim() != 1 or ends.dtype != torch.int32 or ends.device != device:
        raise ValueError("ends must be a 1-D int32 tensor on the rows' device")
    n = ends.shape[0]
    if n > 1 and ends.stride(0) != 1:
        raise ValueError("ends must be contiguous")
    if groups is not None and n != groups:
        raise ValueError("ends and the operands differ in their number of groups")
    return (ends.data_ptr() if n else None), n


def quantize_grouped(x, ends=None, index=None, dual: bool = True, rotate: str = "hadamard",
                     round: str = "rne", seed1: int = 0, seed0: int = 0, sums: bool = False,
                     stream=None) -> GroupedQuantized:
    """Quantize rows that belong to groups, for linear_grouped (see
    mx_quantize_grouped).

    x: 2-D bf16 CUDA rows with ends, the int32 CUDA tensor [groups] of the rows
    behind each group's last (a running sum of the groups' sizes); or 3-D
    [groups, rows, cols], the experts' stacked matrices, without ends. index:
    int32 or int64 [rows], row i is then x[index[i]] (2-D x only; -1 gives zeros).
    dual: also the axis-0 operand, in which every group's rows begin a slice of
    their own. sums: also each group's column sums, fp32 [groups, cols]. Nothing
    waits for the GPU. stream: as for rmsnorm_quantize.
    """
    import torch
    lib = _lib or load_library()
    if x.dtype != torch.bfloat16 or x.dim() not in (2, 3):
        raise ValueError("x must be a 2-D or 3-D bfloat16 tensor")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA (HIP) tensor; there is no CPU path")
    device, each, ep = x.device, -1, None
    if x.dim() == 3:
        if ends is not None or index is not None:
            raise ValueError("stacked matrices take neither ends nor an index")
        groups, each, _ = x.shape
        if groups < 1:
            raise ValueError("x must hold at least one matrix")
        if x.numel() and groups > 1 and x.stride(0) != each * x.stride(1) and each > 1:
            raise ValueError("stacked matrices must follow one another")
        if x.numel() and each == 1:
            x = x[:, 0]
        else:
            x = x.as_strided((groups * each, x.shape[2]), x.stride()[1:])
    else:
        if ends is None:
            raise ValueError("rows need the ends of their groups")
        ep, groups = _ends(ends, None, device)
    src, cols, ld = _source_extents(x)
    rows, ip, bits = src, None, 0
    if index is not None:
        if index.dim() != 1 or index.dtype not in (torch.int32, torch.int64):
            raise ValueError("index must be a 1-D int32 or int64 tensor")
        if index.device != device or (index.shape[0] > 1 and index.stride(0) != 1):
            raise ValueError("index must be contiguous, on the rows' device")
        rows, ip = index.shape[0], index.data_ptr() if index.shape[0] else None
        bits = 64 if index.dtype == torch.int64 else 32
        if rows == 0:
            src, ip = 0, None
    place, handle = _place(device, stream)
    with place:
        size = quantize_grouped_sizes(rows, cols, groups, each, 1)
        if dual:
            size += quantize_grouped_sizes(rows, cols, groups, each, AXIS_GROUPED)
        need = _grouped_workspace(rows, cols, groups, each) if sums else 0
        buf = [torch.empty(b, dtype=torch.uint8, device=device) for b in size]
        ptr = [b.data_ptr() or None for b in buf] + [None, None]
        total = torch.empty((groups, cols), dtype=torch.float32, device=device) if sums else None
        work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        source = GroupedSourceDesc(x.data_ptr() or None, src, cols, ld, ip, bits, rows, groups,
                                   each, ep)
        d1, d0 = GroupedDesc(), GroupedDesc()
        st = lib.mx_quantize_grouped(source, 32, ROTATE[rotate], ROUND[round],
                                     seed1 & 0xFFFFFFFFFFFFFFFF, seed0 & 0xFFFFFFFFFFFFFFFF,
                                     ptr[0], ptr[1], ptr[2], ptr[3],
                                     (total.data_ptr() or None) if sums else None,
                                     work.data_ptr() if need else None, need, d1, d0, handle)
    _check(st, "mx_quantize_grouped")
    q1 = QTensor(buf[0], buf[1], d1.q, groups, each)
    if not dual:
        return GroupedQuantized(q1, None, total)
    if not (rows and cols):     # empty operands have no buffers to tell the call by
        d0.q = QTensorDesc(None, None, rows, cols, AXIS_GROUPED, 32, ROTATE[rotate], ROUND[round],
                           seed0 & 0xFFFFFFFFFFFFFFFF, FORMATS["fp4_e2m1"])
    return GroupedQuantized(q1, QTensor(buf[2], buf[3], d0.q, groups, each), total)


def _matrix(t, name: str, shape, dtype, device):
    """(address, leading dimension) of a matrix of an epilogue, None: none. A
    3-D one (a matrix per group) is its rows one after another."""
    if t is None:
        return None, 0
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must have the output's type, shape and device")
    if t.numel() == 0:
        return None, shape[-1]
    rows, cols = t.shape[-2:]
    if t.stride(-1) != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if len(shape) == 3 and shape[0] > 1:
        if rows > 1 and t.stride(0) != rows * t.stride(1):
            raise ValueError(f"the matrices of {name} must follow one another")
        return t.data_ptr(), t.stride(1) if rows > 1 else t.stride(0)
    return t.data_ptr(), t.stride(-2) if rows > 1 else max(cols, 8 * ((cols + 7) // 8))


def _product(call: str, op: str, A: QTensor, B: QTensor, ends, out_dtype: str, activation: str,
             bias=None, mul=None, residual=None, pre=None, grad: bool = False, dmul=None, out=None,
             stream=None):
    """A product with an epilogue: (C, pre or None, dmul or None). pre: the
    matrix, or whether one is wanted (forward)."""
    import torch
    lib = _lib or load_library()
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[out_dtype]
    device = A.codes.device
    if B.codes.device != device:
        raise ValueError("the operands are on different devices")
    bias_shape = ()
    if ends is None:
        shape = (A.mn, B.mn)
        for q in (A, B):
            if q.desc.axis == AXIS_GROUPED:
                raise ValueError("a grouped operand needs the ends of its groups")
    else:
        if B.groups is None:
            raise ValueError("B must be an operand of grouped rows")
        ep, groups = _ends(ends, B.groups, device)
        bias_shape = (groups,)
        shape = ((groups, A.mn, B.mn) if op == "wgrad"
                 else (A.mn, B.group_rows if op == "fprop" else B.mn))
    n = shape[-1]
    bp, bias_dtype = None, 0
    if bias is not None:
        if tuple(bias.shape) != bias_shape + (n,) or bias.device != device:
            raise ValueError("bias must have a value for each column (of each group)")
        if not bias.is_contiguous():
            raise ValueError("bias must be contiguous")
        bias_dtype, bp = _row_dtype(bias, "bias"), bias.data_ptr() or None
    mp, ldmul = _matrix(mul, "mul", shape, dtype, device)
    rp, ldres = _matrix(residual, "residual", shape, dtype, device)
    place, handle = _place(device, stream)
    with place:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=device)
        cp, ldc = _matrix(out, "out", shape, dtype, device)
        if pre is True:
            pre = torch.empty(shape, dtype=dtype, device=device)
        pre = None if pre is False else pre
        pp, ldpre = _matrix(pre, "pre", shape, dtype, device)
        if grad and mul is not None and dmul is None:
            dmul = torch.empty(shape, dtype=dtype, device=device)
        dp, lddmul = _matrix(dmul, "dmul", shape, dtype, device)
        e = EpilogueDesc(ACTIVATIONS[activation], int(grad), bp, bias_dtype, mp, rp, pp, dp, ldmul,
                         ldres, ldpre, lddmul)
        if ends is None:
            st = lib.mx_linear_fused(OPS[op], A.desc, B.desc, e, cp, ldc, OUT_DTYPES[out_dtype],
                                     handle)
        else:
            da = GroupedDesc(A.desc, A.groups if A.groups is not None else groups, A.group_rows)
            st = lib.mx_linear_grouped(OPS[op], da, GroupedDesc(B.desc, B.groups, B.group_rows),
                                       ep, e, cp, ldc, OUT_DTYPES[out_dtype], handle)
    _check(st, call)
    return out, pre, dmul


def linear_fused(op: str, A: QTensor, B: QTensor, out_dtype: str = "f32", bias=None,
                 activation: str = "none", mul=None, residual=None, save_pre=False, out=None,
                 stream=None):
    """act(A B^T + bias) * mul + residual, one launch (see mx_linear_fused).

    op, A, B, out: as for linear (MXFP4 operands). bias: fp32 or bf16 [N].
    activation: one of ACTIVATIONS. mul, residual: matrices of the output's type
    and shape (row-strided views allowed); either may be out itself, so
    residual=out, out=out adds onto it. save_pre: also return A B^T + bias, in
    the output's type, for linear_act_backward (True, or the matrix to write):
    (C, pre) instead of C. stream: as for rmsnorm_quantize.
    """
    c, pre, _ = _product("mx_linear_fused", op, A, B, None, out_dtype, activation, bias, mul,
                         residual, save_pre, out=out, stream=stream)
    return c if save_pre is False else (c, pre)


def linear_act_backward(A: QTensor, B: QTensor, pre, activation: str, mul=None, ends=None,
                        out_dtype: str = "f32", out=None, dmul=None, stream=None):
    """The gradient of act(pre) * mul taken back through the gate and the
    activation in the epilogue of the product that computes it (see
    mx_linear_fused): with g = linear("dgrad", A, B), returns g * mul *
    act'(pre), the gradient of pre; with mul the pair of it and g * act(pre), the
    gradient of mul. A: q(dY), axis 1; B: q(W), axis 0. With ends (and B from
    quantize_grouped) over experts, as linear_grouped. out may be pre or mul
    itself, dmul too.
    """
    call = "mx_linear_fused" if ends is None else "mx_linear_grouped"
    c, _, dmul = _product(call, "dgrad", A, B, ends, out_dtype, activation, mul=mul, pre=pre,
                          grad=True, dmul=dmul, out=out, stream=stream)
    return c if mul is None else (c, dmul)


def linear_grouped(op: str, A: QTensor, B: QTensor, ends, out_dtype: str = "f32", bias=None,
                   activation: str = "none", mul=None, residual=None, save_pre=False, out=None,
                   stream=None):
    """linear_fused with one matrix per group of rows (the experts of a layer), in
    one launch (see mx_linear_grouped).

    fprop: A = q(X) [T, in] axis 1 (quantize_grouped, quantize or
    rmsnorm_quantize), B = quantize_grouped(W [groups, out, in]).q1 -> [T, out].
    dgrad: A = q(dY) axis 1, B = quantize_grouped(W).q0 -> [T, in]. wgrad: A, B =
    the q0 of quantize_grouped(dY, ends) and quantize_grouped(X, ends) ->
    [groups, out, in]. ends: int32 [groups], the row behind each group's last;
    rows behind the last end are left as they were in out and pre. bias: [groups,
    N]. The rest as for linear_fused.
    """
    c, pre, _ = _product("mx_linear_grouped", op, A, B, ends, out_dtype, activation, bias, mul,
                         residual, save_pre, out=out, stream=stream)
    return c if save_pre is False else (c, pre)
