"""8-bit integer linear layers: a trained gated block as it is served, weights and
activations as integers of 8 bits with one float32 scale a row (a token, or an
output channel).

    q, s = i8_norm(x, w_norm, residual=r)     # s = x + r, and its RMS norm in 8 bits
    h = i8_gated(q, w_gate, w_up)             # silu(q @ w_gate.T) * (q @ w_up.T)
    y = i8_matmul(i8_store(h), w_down)        # exact integer sums, scaled

Weights are :class:`I8` matrices of output channels by inputs, made once with
:func:`i8_store` or from tensors that are there.  Activations are float32 or
bfloat16 CUDA matrices with contiguous rows and any row stride.  The form, the
rounding and the status codes are described in ``include/gemm_f32.h``; as in the
rest of the binding every step runs in the library's CUDA kernels, and there is
no CPU fallback.  These operators serve: results carry no gradient.

``stream`` is as in :mod:`dense_fp32_gemm_row_gb300.q8`.
"""

from __future__ import annotations

import ctypes

import dense_fp32_gemm_row_gb300 as _g
from dense_fp32_gemm_row_gb300 import q8 as _q8

__all__ = [
    "I8", "I8Struct", "TYPE_F32", "TYPE_BF16", "TYPE_I32", "I8_MAX_COLS", "I8_LEAST_EPS",
    "ALGO_I8_PAIR", "ALGO_I8_SINGLE", "ALGO_I8_STREAM", "I8_STREAM_ROWS", "I8_ALGOS",
    "gemm_f32_i8_store", "gemm_f32_i8_norm", "gemm_f32_i8_matmul", "gemm_f32_i8_gated",
    "i8_empty", "i8_store", "i8_norm", "i8_matmul", "i8_gated",
]

TYPE_F32 = 0
TYPE_BF16 = 1
TYPE_I32 = 2
I8_MAX_COLS = 131071
I8_LEAST_EPS = 1e-30
_EPS_TOO_LARGE = 2.0 ** 128 - 2.0 ** 103  # the least number that float32 rounds to an infinity
ALGO_I8_PAIR = 6
ALGO_I8_SINGLE = 7
ALGO_I8_STREAM = 8
I8_STREAM_ROWS = 32
I8_ALGOS = {"auto": 0, "pair": ALGO_I8_PAIR, "single": ALGO_I8_SINGLE, "stream": ALGO_I8_STREAM}


class I8Struct(ctypes.Structure):
    """``gemm_f32_i8`` of the C header."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("ld", ctypes.c_longlong),
                ("rows", ctypes.c_int), ("cols", ctypes.c_int)]

    def __init__(self, codes=None, scales=None, ld=0, rows=0, cols=0):
        super().__init__(codes, scales, ld, _q8._int(rows, "rows"), _q8._int(cols, "cols"))


# ---- raw entry points: addresses and the stream are plain integers --------------------------


def _wide(*values) -> bool:
    """Whether one of them is not what the library's int of 32 bits would get."""
    return any(not -2 ** 31 <= value < 2 ** 31 for value in values)


def gemm_f32_i8_store(X, type, ldx, q, stream=0) -> int:
    if _wide(type):
        return _g.ERR_INVALID_VALUE
    return _g.load().gemm_f32_i8_store(X or None, type, ldx, q, stream or None)


def gemm_f32_i8_norm(X, ldx, R, ldr, W, eps, type, S, lds, q, stream=0) -> int:
    if _wide(type):
        return _g.ERR_INVALID_VALUE
    return _g.load().gemm_f32_i8_norm(X or None, ldx, R or None, ldr, W or None, eps, type, S or None,
                                      lds, q, stream or None)


def gemm_f32_i8_matmul(a, b, Y, type, ldy, algo=0, splits=0, stream=0) -> int:
    if _wide(type, algo, splits):
        return _g.ERR_INVALID_VALUE
    return _g.load().gemm_f32_i8_matmul(a, b, Y or None, type, ldy, algo, splits, stream or None)


def gemm_f32_i8_gated(act, a, gate, up, H, type, ldh, algo=0, splits=0, stream=0) -> int:
    if _wide(act, type, algo, splits):
        return _g.ERR_INVALID_VALUE
    return _g.load().gemm_f32_i8_gated(act, a, gate, up, H or None, type, ldh, algo, splits,
                                       stream or None)


def _declare(lib) -> None:
    vp, i, ll, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    q = ctypes.POINTER(I8Struct)
    lib.gemm_f32_i8_store.argtypes = [vp, i, ll, q, vp]
    lib.gemm_f32_i8_norm.argtypes = [vp, ll, vp, ll, vp, f, i, vp, ll, q, vp]
    lib.gemm_f32_i8_matmul.argtypes = [q, q, vp, i, ll, i, i, vp]
    lib.gemm_f32_i8_gated.argtypes = [i, q, q, q, vp, i, ll, i, i, vp]
    for name in ("store", "norm", "matmul", "gated"):
        getattr(lib, "gemm_f32_i8_" + name).restype = ctypes.c_int


# ---- tensors ---------------------------------------------------------------------------------

_torch = None  # set on first use: importing the package does not import torch
_native = None  # the binding's module for quick calls, where it is built for the installed torch


def _load_torch():
    global _torch, _native
    torch = _q8._torch or _q8._load_torch()
    _native = _q8._native
    if _native is not None:
        lib = _g.load()
        _native.bind_i8(*(ctypes.cast(getattr(lib, "gemm_f32_i8_" + name), ctypes.c_void_p).value
                          for name in ("store", "norm", "matmul", "gated")), I8)
    _torch = torch
    return torch


def _layout(codes, scales, cols):
    """(device, rows, row stride) of a matrix's two tensors, which are checked."""
    if (codes.dtype is not _torch.int8 or scales.dtype is not _torch.float32 or codes.dim() != 2
            or scales.dim() != 1 or not codes.is_cuda):
        raise ValueError("codes must be a 2-D int8 and scales a 1-D float32 CUDA tensor")
    _q8._as_stored(codes, "codes")
    _q8._as_stored(scales, "scales")
    device = codes.get_device()
    if scales.get_device() != device:
        raise ValueError("codes and scales must be on one device")
    rows, width = codes.shape
    _q8._int(rows, "the rows of codes")
    _q8._int(cols, "cols")
    if cols < 0 or width < cols or scales.shape[0] != rows:
        raise ValueError("codes must be (rows, >= cols) and scales (rows,)")
    ld, one = codes.stride()
    if rows <= 1:
        ld = (width + 15) & ~15
    if rows and cols:
        if (one != 1 and width > 1) or ld < cols or (codes.data_ptr() | ld) & 15:
            raise ValueError("codes must have contiguous rows, a 16-byte aligned base and a row "
                             "stride that is a multiple of 16")
        if rows > 1 and scales.stride()[0] != 1:
            raise ValueError("scales must be contiguous")
        if (codes.storage_offset() + (rows - 1) * ld + cols > codes.untyped_storage().nbytes()
                or 4 * (scales.storage_offset() + rows) > scales.untyped_storage().nbytes()):
            raise ValueError("codes and scales must have their memory")
    return device, rows, ld


class I8:
    """A ``rows`` x ``cols`` matrix of 8-bit integers with a scale a row.

    ``codes`` is a (rows, >= cols) int8 and ``scales`` a (rows,) float32 CUDA
    tensor; ``codes`` starts on a 16-byte boundary and has a row stride that is a
    multiple of 16.  A call reads or writes the memory that these tensors have at
    that time, and is refused when they no longer hold the matrix.
    """

    __slots__ = ("codes", "scales", "cols")

    def __init__(self, codes, scales, cols):
        if _torch is None:
            _load_torch()
        if _native is None or not _native.i8_fits(codes, scales, cols):
            _layout(codes, scales, cols)
        self.codes, self.scales, self.cols = codes, scales, cols

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def device(self) -> int:
        """The index of the CUDA device."""
        return self.codes.get_device()

    @property
    def struct(self) -> I8Struct:
        """The matrix for the raw entry points; valid as long as the memory its tensors have now."""
        _, rows, ld = _layout(self.codes, self.scales, self.cols)
        return I8Struct(self.codes.data_ptr(), self.scales.data_ptr(), ld, rows, self.cols)

    @property
    def nbytes(self) -> int:
        """Bytes that the two tensors hold."""
        return self.codes.numel() + 4 * self.scales.numel()

    def record_stream(self, stream) -> None:
        """As ``torch.Tensor.record_stream``, for a matrix used on another stream."""
        self.codes.record_stream(stream)
        self.scales.record_stream(stream)

    def __repr__(self):
        return f"I8({self.rows} x {self.cols})"


def _make(rows, cols, device) -> I8:
    """An uninitialised matrix, its rows padded to 16 bytes."""
    q = I8.__new__(I8)
    device = f"cuda:{device}"
    q.codes = _torch.empty((rows, (cols + 15) & ~15), dtype=_torch.int8, device=device)
    q.scales = _torch.empty((rows,), dtype=_torch.float32, device=device)
    q.cols = cols
    return q


def _type(dtype, what, whole=False) -> int:
    if dtype is _torch.float32:
        return TYPE_F32
    if dtype is _torch.bfloat16:
        return TYPE_BF16
    if whole and dtype is _torch.int32:
        return TYPE_I32
    raise ValueError(f"{what} is torch.float32{', torch.int32' if whole else ''} or "
                     f"torch.bfloat16, not {dtype}")


def _matrix(t, what):
    """(rows, cols, row stride) of a float32 or bfloat16 CUDA matrix with contiguous rows."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D CUDA tensor")
    return _q8._strides(t, what)


def _like(t, rows, cols, dtype, device, what):
    """The row stride of a given operand, which must be rows x cols of ``dtype`` on ``device``."""
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype}, not {t.dtype}")
    r, c, ld = _matrix(t, what)
    if r != rows or c != cols:
        raise ValueError(f"{what} must be {rows} x {cols}, not {r} x {c}")
    _on(t.get_device(), device)
    return ld


def _on(device, other):
    if device != other:
        raise ValueError("all tensors must be on one device")


def _given(q, rows, cols, device, what) -> I8:
    if q.rows != rows or q.cols != cols:
        raise ValueError(f"{what} must hold {rows} x {cols}, not {q.rows} x {q.cols}")
    _on(q.device, device)
    return q


def i8_empty(rows, cols, device="cuda") -> I8:
    """An uninitialised rows x cols matrix."""
    torch = _torch or _load_torch()
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("an 8-bit matrix is made on a CUDA device")
    if _q8._int(rows, "rows") < 0 or _q8._int(cols, "cols") < 0:
        raise ValueError("rows and cols must not be negative")
    with torch.cuda.device(device):
        return _make(rows, cols, torch.cuda.current_device())


def i8_store(x, out=None, stream=None) -> I8:
    """The rows of ``x`` (float32 or bfloat16) in 8 bits, in ``out`` if given."""
    if _torch is None:
        _load_torch()
    if out is None and stream is None and _native is not None:
        q = _native.i8_store(x)
        if q is not None:
            return q
    code = _type(x.dtype, "x's type")
    rows, cols, ld = _matrix(x, "x")
    device = x.get_device()
    if stream is not None or _q8._away(device):
        return _q8._elsewhere(lambda: i8_store(x, out), device, stream, (x, out))
    q = _make(rows, cols, device) if out is None else _given(out, rows, cols, device, "out")
    st = _q8._lib.gemm_f32_i8_store(x.data_ptr(), code, ld, q.struct, _q8._stream_of(device))
    if st:
        _g.check(st, "i8_store")
    return q


def i8_norm(x, weight, residual=None, eps=1e-6, out=None, total=None, stream=None):
    """``s = x + residual`` and its root-mean-square norm times ``weight`` in 8 bits: ``(q, s)``.

    All are of one type, float32 or bfloat16.  Without ``residual`` the norm is
    that of ``x``, and ``s`` is None.  ``out`` and ``total`` may be given for the
    two results; neither may share memory with an operand.
    """
    if _torch is None:
        _load_torch()
    if out is None and total is None and stream is None and _native is not None:
        made = _native.i8_norm(x, weight, residual, eps)
        if made is not None:
            return made
    code = _type(x.dtype, "x's type")
    rows, cols, ldx = _matrix(x, "x")
    device = x.get_device()
    if weight.dtype is not x.dtype or weight.dim() != 1 or weight.shape[0] != cols:
        raise ValueError(f"weight must be ({cols},) of x's type")
    if cols > 1 and weight.stride()[0] != 1:
        raise ValueError("weight must be contiguous")
    _q8._as_stored(weight, "weight")
    _on(weight.get_device(), device)
    ldr = 0 if residual is None else _like(residual, rows, cols, x.dtype, device, "residual")
    if total is not None and residual is None:
        raise ValueError("total is x + residual: it needs residual")
    if not I8_LEAST_EPS <= eps < _EPS_TOO_LARGE:
        raise ValueError("eps must be at least 1e-30 and finite in float32")
    if stream is not None or _q8._away(device):
        return _q8._elsewhere(lambda: i8_norm(x, weight, residual, eps, out, total), device, stream,
                              (x, weight, residual, out, total))
    if residual is None:
        s, lds = None, 0
    elif total is None:
        s, lds = _torch.empty((rows, cols), dtype=x.dtype, device=x.device), cols or 1
    else:
        s, lds = total, _like(total, rows, cols, x.dtype, device, "total")
    q = _make(rows, cols, device) if out is None else _given(out, rows, cols, device, "out")
    st = _q8._lib.gemm_f32_i8_norm(
        x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
        weight.data_ptr(), eps, code, None if s is None else s.data_ptr(), lds, q.struct,
        _q8._stream_of(device))
    if st:
        _g.check(st, "i8_norm")
    return q, s


def _output(a, w, dtype, out):
    """The output of a product, its row stride."""
    if out is None:
        return _torch.empty((a.rows, w.rows), dtype=dtype, device=a.codes.device), w.rows or 1
    return out, _like(out, a.rows, w.rows, dtype, a.device, "out")


def _inputs(a, w):
    if a.cols != w.cols:
        raise ValueError(f"tokens of {a.cols} columns, weights of {w.cols}")
    if a.cols > I8_MAX_COLS:
        raise ValueError(f"sums over more than {I8_MAX_COLS} columns may overflow 32 bits")
    _on(w.device, a.device)


def i8_matmul(a, w, dtype=None, out=None, algo="auto", splits=0, stream=None):
    """``a @ w.T`` of tokens ``a`` and weights ``w`` (channels, inputs), both :class:`I8`.

    The sums over codes are exact; ``dtype`` is float32 (the default) or
    bfloat16 for their values, or int32 for the sums themselves.  ``algo``
    ("pair" or "single" CTAs a tile, or "stream" for at most 32 tokens) and
    ``splits`` (of single CTAs' tiles, over K) are chosen by size; results do not
    depend on them.
    """
    torch = _torch or _load_torch()
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    code = _type(dtype, "dtype", whole=True)
    if out is None and stream is None and algo == "auto" and splits == 0 and _native is not None:
        y = _native.i8_matmul(a, w, code)
        if y is not None:
            return y
    which = _q8._name(I8_ALGOS, algo, "algo")
    _q8._int(splits, "splits")
    _inputs(a, w)
    device = a.device
    if stream is not None or _q8._away(device):
        return _q8._elsewhere(lambda: i8_matmul(a, w, dtype, out, algo, splits), device, stream, (a, w, out))
    qa, qw = a.struct, w.struct
    y, ldy = _output(a, w, dtype, out)
    st = _q8._lib.gemm_f32_i8_matmul(qa, qw, y.data_ptr(), code, ldy, which, splits,
                                     _q8._stream_of(device))
    if st:
        _g.check(st, "i8_matmul")
    return y


def i8_gated(a, gate, up, act="silu", dtype=None, out=None, algo="auto", splits=0, stream=None):
    """``act(a @ gate.T) * (a @ up.T)`` of tokens ``a`` and two weights, all :class:`I8`, as
    float32 (the default) or bfloat16; ``act`` is "silu" or "gelu", ``algo`` and ``splits`` are as
    for :func:`i8_matmul`."""
    torch = _torch or _load_torch()
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    code = _type(dtype, "dtype")
    which = _q8._name(_q8.ACTS, act, "act")
    if out is None and stream is None and algo == "auto" and splits == 0 and _native is not None:
        h = _native.i8_gated(a, gate, up, which, code)
        if h is not None:
            return h
    how = _q8._name(I8_ALGOS, algo, "algo")
    _q8._int(splits, "splits")
    _inputs(a, gate)
    _given(up, gate.rows, gate.cols, a.device, "up")
    device = a.device
    if stream is not None or _q8._away(device):
        return _q8._elsewhere(lambda: i8_gated(a, gate, up, act, dtype, out, algo, splits), device,
                              stream, (a, gate, up, out))
    qa, qg, qu = a.struct, gate.struct, up.struct
    h, ldh = _output(a, gate, dtype, out)
    st = _q8._lib.gemm_f32_i8_gated(which, qa, qg, qu, h.data_ptr(), code, ldh, how,
                                    splits, _q8._stream_of(device))
    if st:
        _g.check(st, "i8_gated")
    return h
