"""8-bit activation checkpoints: what a training step keeps of a layer between
its forward and its backward pass, a byte an element, and the operators of the
backward pass that read it in that form.

    q = q8_store(x)                        # x: (tokens, features) float32
    x_hat = q8_restore(q)                  # float32, or dtype=torch.bfloat16
    dw = q8_wgrad(q, dy)                   # x_hat.T @ dy, without x_hat
    h, gq, uq = q8_gated(gate, up)         # h = silu(gate) * up
    dgate, dup, hq = q8_gated_backward(gq, uq, dh)

Tensors are float32 CUDA matrices with contiguous rows and any row stride, so
that the halves of one wider product need no copy.  The format, the layout of
a :class:`Q8`'s two byte tensors and the status codes are described in
``include/gemm_f32.h``; as in the rest of the binding every step runs in the
library's CUDA kernels, and there is no CPU fallback.

``stream`` (a ``torch.cuda.Stream``, default the current one) is where a call
runs; with a stream other than the current one the caller orders it against
the work that made the inputs, and the tensors are kept from being reused by
the allocator before the call has run.
"""

from __future__ import annotations

import ctypes

import dense_fp32_gemm_row_gb300 as _g

__all__ = [
    "Q8", "Q8Struct", "Q8_INT8", "Q8_E4M3", "Q8_FORMATS", "Q8_BLOCK", "Q8_TO_F32", "Q8_TO_BF16",
    "ACT_SILU", "ACT_GELU", "ACTS", "ALGO_3XBF16",
    "ALGO_3XBF16_PAIR", "ALGO_3XBF16_SINGLE", "Q8_ALGOS", "gemm_f32_q8_store", "gemm_f32_q8_restore",
    "gemm_f32_q8_wgrad", "gemm_f32_q8_gated", "gemm_f32_q8_gated_backward", "q8_empty",
    "q8_store", "q8_restore", "q8_wgrad", "q8_gated", "q8_gated_backward",
]

Q8_INT8 = 0
Q8_E4M3 = 1
Q8_FORMATS = {"int8": Q8_INT8, "e4m3": Q8_E4M3}
_FORMAT_NAMES = {value: name for name, value in Q8_FORMATS.items()}
Q8_BLOCK = 32
Q8_TO_F32 = 0
Q8_TO_BF16 = 1
ACT_SILU = 0
ACT_GELU = 1
ALGO_3XBF16 = 3
ALGO_3XBF16_PAIR = 4
ALGO_3XBF16_SINGLE = 5
Q8_ALGOS = {"auto": 0, "ffma": 1, "3xbf16": ALGO_3XBF16, "3xbf16_pair": ALGO_3XBF16_PAIR,
            "3xbf16_single": ALGO_3XBF16_SINGLE}
ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU}


_INT_MAX = 2 ** 31 - 1  # ctypes passes on the low 32 bits of an int that is larger


def _int(value, what):
    """``value``, which the library takes as an int of 32 bits."""
    if not -_INT_MAX <= value <= _INT_MAX:
        raise ValueError(f"{what} must be below 2^31, not {value}")
    return value


class Q8Struct(ctypes.Structure):
    """``gemm_f32_q8`` of the C header."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ldcodes", ctypes.c_longlong), ("ldscales", ctypes.c_longlong),
                ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("format", ctypes.c_int)]

    def __init__(self, codes=None, scales=None, ldcodes=0, ldscales=0, rows=0, cols=0, format=0):
        super().__init__(codes, scales, ldcodes, ldscales, _int(rows, "rows"), _int(cols, "cols"),
                         format)


# ---- raw entry points: addresses and the stream are plain integers --------------------------


def gemm_f32_q8_store(X, ldx, q, stream=0) -> int:
    return _g.load().gemm_f32_q8_store(X or None, ldx, q, stream or None)


def gemm_f32_q8_restore(q, X, ldx, type=Q8_TO_F32, stream=0) -> int:
    return _g.load().gemm_f32_q8_restore(q, X or None, ldx, type, stream or None)


def gemm_f32_q8_wgrad(x, dY, lddy, N, alpha, beta, dW, lddw, algo=0, splits=0, stream=0) -> int:
    if abs(N) > _INT_MAX or abs(splits) > _INT_MAX:
        return _g.ERR_INVALID_VALUE
    return _g.load().gemm_f32_q8_wgrad(x, dY or None, lddy, N, alpha, beta, dW or None, lddw, algo,
                                       splits, stream or None)


def gemm_f32_q8_gated(act, G, ldg, U, ldu, H, ldh, gq, uq, stream=0) -> int:
    return _g.load().gemm_f32_q8_gated(act, G or None, ldg, U or None, ldu, H or None, ldh, gq, uq,
                                       stream or None)


def gemm_f32_q8_gated_backward(act, gq, uq, dH, lddh, dG, lddg, dU, lddu, hq=None,
                               stream=0) -> int:
    return _g.load().gemm_f32_q8_gated_backward(act, gq, uq, dH or None, lddh, dG or None, lddg,
                                                dU or None, lddu, hq, stream or None)


def _declare(lib) -> None:
    vp, i, ll, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
    q = ctypes.POINTER(Q8Struct)
    lib.gemm_f32_q8_store.argtypes = [vp, ll, q, vp]
    lib.gemm_f32_q8_restore.argtypes = [q, vp, ll, i, vp]
    lib.gemm_f32_q8_wgrad.argtypes = [q, vp, ll, i, f, f, vp, ll, i, i, vp]
    lib.gemm_f32_q8_gated.argtypes = [i, vp, ll, vp, ll, vp, ll, q, q, vp]
    lib.gemm_f32_q8_gated_backward.argtypes = [i, q, q, vp, ll, vp, ll, vp, ll, q, vp]
    for name in ("store", "restore", "wgrad", "gated", "gated_backward"):
        getattr(lib, "gemm_f32_q8_" + name).restype = ctypes.c_int


# ---- tensors ---------------------------------------------------------------------------------
#
# A small call takes the GPU a few microseconds, so what the binding spends on the host is most
# of it.  The ordinary call -- plain tensors on the current device, nothing given for its results --
# is one call of the module built from csrc/binding/tensors.cpp, which answers None to anything
# else; what follows here then looks at the operands one by one, and finds the error if there is one.

_torch = None  # set on first use: importing the package does not import torch
_stream_of = _lib = None
_native = None  # the module, where it is built for the installed torch
_one_device = True


def _load_torch():
    global _torch, _stream_of, _lib, _native, _one_device
    import torch

    # the function behind torch.cuda.current_stream
    _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream",
                         lambda index: torch.cuda.current_stream(index).cuda_stream)
    _lib = _g.load()
    try:
        from dense_fp32_gemm_row_gb300 import _tensors

        _tensors.bind(*(ctypes.cast(getattr(_lib, "gemm_f32_q8_" + name), ctypes.c_void_p).value
                        for name in ("store", "restore", "wgrad", "gated", "gated_backward")),
                      _g.check, Q8, str(torch.__version__))
        _native = _tensors
    except ImportError:  # not built, or for another torch
        _native = None
    _one_device = torch.cuda.device_count() <= 1
    _torch = torch
    return torch


def _layout(codes, scales, cols):
    """(device, rows, row strides) of a checkpoint's two tensors, which are checked."""
    if (codes.dtype is not _torch.uint8 or scales.dtype is not _torch.uint8 or codes.dim() != 2
            or scales.dim() != 2 or not codes.is_cuda):
        raise ValueError("codes and scales must be 2-D uint8 CUDA tensors")
    if scales.get_device() != codes.get_device():
        raise ValueError("codes and scales must be on one device")
    (rows, width), (rows2, width2) = codes.shape, scales.shape
    blocks = (cols + 31) >> 5
    _int(rows, "the rows of codes")
    _int(cols, "cols")
    if cols < 0 or rows2 != rows or width < cols or width2 < blocks:
        raise ValueError("codes must be (rows, >= cols), scales (rows, >= ceil(cols / 32))")
    (ldc, one), (lds, one2) = codes.stride(), scales.stride()
    if rows <= 1:
        ldc, lds = (width + 15) & ~15, (width2 + 15) & ~15
    if rows and cols:
        if (one != 1 or one2 != 1 or ldc < cols or lds < blocks
                or (codes.data_ptr() | scales.data_ptr() | ldc | lds) & 15):
            raise ValueError("codes and scales must have contiguous rows, 16-byte aligned bases "
                             "and row strides that are multiples of 16")
        for t, ld, n in ((codes, ldc, cols), (scales, lds, blocks)):
            if t.storage_offset() + (rows - 1) * ld + n > t.untyped_storage().nbytes():
                raise ValueError("codes and scales must have their memory")
    return codes.get_device(), rows, ldc, lds


class _Held:
    """Two tensors and their layout, as the module's objects of this name hold them."""

    __slots__ = ("_tensors", "device", "rows", "cols", "format", "ldcodes", "ldscales")

    def __init__(self, codes, scales, cols, format):
        self._tensors = codes, scales
        self.cols, self.format = cols, format
        self.device, self.rows, self.ldcodes, self.ldscales = _layout(codes, scales, cols)

    def tensors(self):
        return self._tensors

    # whoever has the tensors can give them other memory: looked at again for every call
    @property
    def codes(self):
        layout = self.device, self.rows, self.ldcodes, self.ldscales
        if _layout(*self._tensors, self.cols) != layout:
            raise ValueError("the checkpoint's tensors no longer hold it")
        return self._tensors[0].data_ptr()

    @property
    def scales(self):
        return self._tensors[1].data_ptr()


def _empty(rows, cols, bf16, device):
    if _native is not None:
        return _native.empty(rows, cols, bf16, device)
    return _torch.empty((rows, cols), dtype=_torch.bfloat16 if bf16 else _torch.float32,
                        device=f"cuda:{device}")


def _make(device, rows, cols, format) -> Q8:
    """An uninitialised checkpoint: rows of codes and of exponents, each padded to 16 bytes."""
    if _native is not None:
        return _native.make(rows, cols, Q8_FORMATS[format], device)
    ldc, lds = (cols + 15) & ~15, (((cols + 31) >> 5) + 15) & ~15
    codes, scales = (_torch.empty((rows, ld), dtype=_torch.uint8, device=f"cuda:{device}")
                     for ld in (ldc, lds))
    q = Q8.__new__(Q8)
    q._held = _Held(codes, scales, cols, Q8_FORMATS[format])
    return q


def _name(table, value, what):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{what} is one of {', '.join(table)}, not {value!r}") from None


class Q8:
    """An 8-bit checkpoint of a ``rows`` x ``cols`` matrix.

    ``codes`` is a (rows, >= cols) and ``scales`` a (rows, >= ceil(cols / 32))
    uint8 CUDA tensor; both start on 16-byte boundaries and have row strides
    that are multiples of 16.  ``format`` is "int8" or "e4m3".  A call reads or
    writes the memory that these tensors have at that time, and is refused when
    it has become too small.
    """

    __slots__ = ("_held",)

    def __init__(self, codes, scales, cols, format="int8"):
        if _torch is None:
            _load_torch()
        fmt = _name(Q8_FORMATS, format, "format")
        if _native is not None:
            self._held = _native.wrap(codes, scales, cols, fmt)
            if self._held is not None:
                return
        self._held = _Held(codes, scales, cols, fmt)

    rows = property(lambda self: self._held.rows)
    cols = property(lambda self: self._held.cols)
    format = property(lambda self: _FORMAT_NAMES[self._held.format])
    device = property(lambda self: self._held.device, doc="The index of the CUDA device.")

    @property
    def codes(self):
        """The code bytes, (rows, cols rounded up to 16) for a checkpoint made here."""
        return self._held.tensors()[0]

    @property
    def scales(self):
        """The exponent bytes, one for each block of 32 columns."""
        return self._held.tensors()[1]

    @property
    def struct(self) -> Q8Struct:
        """The checkpoint for the raw entry points; valid as long as this object and the memory its
        tensors have now."""
        h = self._held
        return Q8Struct(h.codes, h.scales, h.ldcodes, h.ldscales, h.rows, h.cols, h.format)

    @property
    def nbytes(self) -> int:
        """Bytes that the two tensors hold."""
        return self.codes.numel() + self.scales.numel()

    def record_stream(self, stream) -> None:
        """As ``torch.Tensor.record_stream``, for a checkpoint used on another stream."""
        for t in self._held.tensors():
            t.record_stream(stream)

    def __repr__(self):
        return f"Q8({self.rows} x {self.cols}, {self.format})"


def _matrix(t, what):
    """(rows, cols, row stride) of a float32 CUDA matrix with contiguous rows."""
    if t.dtype is not _torch.float32 or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D float32 CUDA tensor")
    return _strides(t, what)


def _strides(t, what):
    rows, cols = t.shape
    if rows > _INT_MAX or cols > _INT_MAX:
        raise ValueError(f"{what} must have fewer than 2^31 rows and columns, not {rows} x {cols}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1 and rows:
        raise ValueError(f"{what} must have contiguous rows")
    if rows <= 1:
        return rows, cols, cols or 1
    if s0 < cols or s0 < 1:
        raise ValueError(f"{what} must have rows that do not overlap")
    return rows, cols, s0


def _like(t, rows, cols, device, what):
    """The row stride of a given float32 operand, which must be rows x cols on ``device``."""
    r, c, ld = _matrix(t, what)
    if r != rows or c != cols:
        raise ValueError(f"{what} must be {rows} x {cols}, not {r} x {c}")
    if t.get_device() != device:
        raise ValueError("all tensors must be on one device")
    return ld


def _given(q, rows, cols, format, device, what) -> Q8:
    """A checkpoint given for a result, or for an operand of this shape."""
    if q.rows != rows or q.cols != cols:
        raise ValueError(f"{what} must hold {rows} x {cols}, not {q.rows} x {q.cols}")
    if q.format != format:
        raise ValueError(f"{what} must be in {format}, not {q.format}")
    if q.device != device:
        raise ValueError("all tensors must be on one device")
    return q


def _elsewhere(call, device, stream, tensors):
    """``call()`` on ``device`` and ``stream``, whose results then belong to that stream, with the
    tensors it reads or writes kept from reuse until it has run.  None: nothing to switch."""
    torch = _torch
    if stream is not None and stream.device.index != device:
        raise ValueError("the stream must be on the tensors' device")
    if stream is not None and stream != torch.cuda.current_stream(device):
        with torch.cuda.stream(stream):
            result = call()
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return result
    with torch.cuda.device(device):
        return call()


def _away(device) -> bool:
    return not _one_device and device >= 0 and device != _torch.cuda.current_device()


def q8_empty(rows, cols, format="int8", device="cuda") -> Q8:
    """An uninitialised checkpoint of a rows x cols matrix."""
    torch = _torch or _load_torch()
    _name(Q8_FORMATS, format, "format")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("a checkpoint is made on a CUDA device")
    _int(rows, "rows")
    _int(cols, "cols")
    with torch.cuda.device(device):
        return _make(torch.cuda.current_device(), rows, cols, format)


def q8_store(x, format="int8", out=None, stream=None) -> Q8:
    """The 8-bit checkpoint of ``x`` (rows, cols), in ``out`` if given."""
    if _torch is None:
        _load_torch()
    fmt = _name(Q8_FORMATS, format, "format")
    if out is None and stream is None and _native is not None:
        q = _native.store(x, fmt)
        if q is not None:
            return q
    rows, cols, ld = _matrix(x, "x")
    device = x.get_device()
    if stream is not None or _away(device):
        return _elsewhere(lambda: q8_store(x, format, out), device, stream, (x, out))
    q = _make(device, rows, cols, format) if out is None else _given(out, rows, cols, format, device,
                                                                     "out")
    st = _lib.gemm_f32_q8_store(x.data_ptr(), ld, q.struct, _stream_of(device))
    if st:
        _g.check(st, "q8_store")
    return q


def q8_restore(q, out=None, dtype=None, stream=None):
    """The values ``q`` stands for, as float32 or (``dtype=torch.bfloat16``) bfloat16, both exact."""
    torch = _torch or _load_torch()
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise ValueError("dtype is torch.float32 or torch.bfloat16")
    if out is None and stream is None and _native is not None:
        x = _native.restore(q._held, dtype is torch.bfloat16)
        if x is not None:
            return x
    device = q.device
    if stream is not None or _away(device):
        return _elsewhere(lambda: q8_restore(q, out, dtype), device, stream, (q, out))
    if out is None:
        rows, cols = q.rows, q.cols
        x = _empty(rows, cols, dtype is torch.bfloat16, device)
        ld = cols or 1
    else:
        x = out
        if x.dtype is not dtype or x.dim() != 2 or x.get_device() != device:
            raise ValueError(f"out must be a 2-D {dtype} tensor on the checkpoint's device")
        rows, cols, ld = _strides(x, "out")
        if rows != q.rows or cols != q.cols:
            raise ValueError(f"out must be {q.rows} x {q.cols}, not {rows} x {cols}")
    st = _lib.gemm_f32_q8_restore(q.struct, x.data_ptr(), ld,
                                  Q8_TO_F32 if dtype is torch.float32 else Q8_TO_BF16,
                                  _stream_of(device))
    if st:
        _g.check(st, "q8_restore")
    return x


def q8_wgrad(q, dy, out=None, alpha=1.0, beta=0.0, algo="auto", splits=0, stream=None):
    """``out = alpha * x_hat.T @ dy + beta * out`` from the checkpoint ``q`` of x.

    ``dy`` is (q.rows, N); ``out`` (q.cols, N) is allocated if not given, and
    must be given for ``beta`` other than 0 (gradient accumulation).  ``algo``
    is "auto", "ffma" or "3xbf16" (the tensor-core kernel; "3xbf16_pair" and
    "3xbf16_single" force its tiles), ``splits`` the number of ranges the
    latter splits the tokens into (0: chosen by size).  "ffma" sums with
    rounding to nearest; the tensor core truncates (relative errors of 4e-7 up
    to 512 tokens and 7e-7 beyond, nearly all towards zero).
    """
    if _torch is None:
        _load_torch()
    if (out is None and stream is None and _native is not None and algo == "auto" and splits == 0
            and alpha == 1.0 and beta == 0.0):
        dw = _native.wgrad(q._held, dy)
        if dw is not None:
            return dw
    rows, N, ldy = _matrix(dy, "dy")
    if rows != q.rows:
        raise ValueError(f"dy must have {q.rows} rows, not {rows}")
    code = _name(Q8_ALGOS, algo, "algo")
    _int(splits, "splits")
    device = q.device
    if dy.get_device() != device:
        raise ValueError("all tensors must be on one device")
    if stream is not None or _away(device):
        return _elsewhere(lambda: q8_wgrad(q, dy, out, alpha, beta, algo, splits), device, stream,
                          (q, dy, out))
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out, the gradient to add to")
        dw, ldw = _empty(q.cols, N, 0, device), N or 1
    else:
        dw, ldw = out, _like(out, q.cols, N, device, "out")
    st = _lib.gemm_f32_q8_wgrad(q.struct, dy.data_ptr(), ldy, N, alpha, beta, dw.data_ptr(), ldw,
                                code, splits, _stream_of(device))
    if st:
        _g.check(st, "q8_wgrad")
    return dw


def q8_gated(gate, up, act="silu", format="int8", out=None, gate_q=None, up_q=None, stream=None):
    """``h = act(gate) * up`` and the checkpoints of gate and up: ``(h, gate_q, up_q)``.

    Two checkpoints made here may lie in one allocation, which is given back when both are gone
    (and with it ``record_stream`` of one holds the other's memory too); made with
    :func:`q8_empty` and given as ``gate_q`` and ``up_q`` they are apart.
    """
    if _torch is None:
        _load_torch()
    code = _name(ACTS, act, "act")
    fmt = _name(Q8_FORMATS, format, "format")
    if out is None and gate_q is None and up_q is None and stream is None and _native is not None:
        made = _native.gated(gate, up, code, fmt)
        if made is not None:
            return made
    rows, cols, ldg = _matrix(gate, "gate")
    device = gate.get_device()
    ldu = _like(up, rows, cols, device, "up")
    if stream is not None or _away(device):
        return _elsewhere(lambda: q8_gated(gate, up, act, format, out, gate_q, up_q), device,
                          stream, (gate, up, out, gate_q, up_q))
    if out is None:
        h, ldh = _empty(rows, cols, 0, device), cols or 1
    else:
        h, ldh = out, _like(out, rows, cols, device, "out")
    gq, uq = (_make(device, rows, cols, format) if q is None else
              _given(q, rows, cols, format, device, what)
              for q, what in ((gate_q, "gate_q"), (up_q, "up_q")))
    st = _lib.gemm_f32_q8_gated(code, gate.data_ptr(), ldg, up.data_ptr(), ldu, h.data_ptr(), ldh,
                                gq.struct, uq.struct, _stream_of(device))
    if st:
        _g.check(st, "q8_gated")
    return h, gq, uq


def q8_gated_backward(gate_q, up_q, dh, act="silu", dgate=None, dup=None, h_q=None,
                      want_h=True, stream=None):
    """The gradients of a gated unit from its checkpoints: ``(dgate, dup, h_q)``.

    ``h_q`` is the checkpoint of ``act(gate) * up`` as recomputed from them,
    for the weight gradient of the layer that follows; None if ``want_h`` is
    false.  ``dgate`` and ``dup`` may be given, for instance as the halves of
    one buffer.
    """
    if _torch is None:
        _load_torch()
    code = _name(ACTS, act, "act")
    if dgate is None and dup is None and h_q is None and stream is None and _native is not None:
        made = _native.gated_backward(gate_q._held, up_q._held, dh, code, 1 if want_h else 0)
        if made is not None:
            return made
    rows, cols, format, device = gate_q.rows, gate_q.cols, gate_q.format, gate_q.device
    _given(up_q, rows, cols, format, device, "up_q")
    ldh = _like(dh, rows, cols, device, "dh")
    if h_q is not None and not want_h:
        raise ValueError("h_q given, and want_h false")
    if stream is not None or _away(device):
        return _elsewhere(lambda: q8_gated_backward(gate_q, up_q, dh, act, dgate, dup, h_q, want_h),
                          device, stream, (gate_q, up_q, dh, dgate, dup, h_q))
    if dgate is None:
        dg, ldg = _empty(rows, cols, 0, device), cols or 1
    else:
        dg, ldg = dgate, _like(dgate, rows, cols, device, "dgate")
    if dup is None:
        du, ldu = _empty(rows, cols, 0, device), cols or 1
    else:
        du, ldu = dup, _like(dup, rows, cols, device, "dup")
    if h_q is not None:
        _given(h_q, rows, cols, format, device, "h_q")
    elif want_h:
        h_q = _make(device, rows, cols, format)
    st = _lib.gemm_f32_q8_gated_backward(code, gate_q.struct, up_q.struct, dh.data_ptr(), ldh,
                                         dg.data_ptr(), ldg, du.data_ptr(), ldu,
                                         None if h_q is None else h_q.struct,
                                         _stream_of(device))
    if st:
        _g.check(st, "q8_gated_backward")
    return dg, du, h_q
