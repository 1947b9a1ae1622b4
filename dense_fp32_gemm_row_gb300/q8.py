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


class Q8Struct(ctypes.Structure):
    """``gemm_f32_q8`` of the C header."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ldcodes", ctypes.c_longlong), ("ldscales", ctypes.c_longlong),
                ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("format", ctypes.c_int)]


# ---- raw entry points: addresses and the stream are plain integers --------------------------


def gemm_f32_q8_store(X, ldx, q, stream=0) -> int:
    return _g.load().gemm_f32_q8_store(X or None, ldx, q, stream or None)


def gemm_f32_q8_restore(q, X, ldx, type=Q8_TO_F32, stream=0) -> int:
    return _g.load().gemm_f32_q8_restore(q, X or None, ldx, type, stream or None)


def gemm_f32_q8_wgrad(x, dY, lddy, N, alpha, beta, dW, lddw, algo=0, splits=0, stream=0) -> int:
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
# of it: a call looks at each tensor once and takes the slower ways (another stream, another
# device) only where they are needed.  Making a tensor by torch.empty costs more than the launch
# (see csrc/binding/tensors.cpp, which makes the outputs where it is built); memory alone from the
# same allocator takes 0.6 us, so a checkpoint holds that and makes its two tensors when they are
# asked for.

_torch = None  # set on first use: importing the package does not import torch
_stream_of = _alloc = _free = _empty = _lib = None
_one_device = True


def _load_torch():
    global _torch, _stream_of, _alloc, _free, _empty, _lib, _one_device
    import torch

    # the functions behind torch.cuda's current_stream, caching_allocator_alloc and _delete
    _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream",
                         lambda index: torch.cuda.current_stream(index).cuda_stream)
    _alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc",
                     lambda size, stream: torch.cuda.caching_allocator_alloc(size, None, stream))
    _free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete",
                    torch.cuda.caching_allocator_delete)
    try:
        from dense_fp32_gemm_row_gb300._tensors import empty as _empty
    except ImportError:  # not built, or for another torch
        def _empty(rows, cols, bf16, device):
            return torch.empty((rows, cols), dtype=torch.bfloat16 if bf16 else torch.float32,
                               device=device)
    _lib = _g.load()
    _one_device = torch.cuda.device_count() <= 1
    _torch = torch
    return torch


class _Memory:
    """Bytes of torch's caching allocator for the current stream, freed with this object."""

    __slots__ = ("address", "size", "device", "stream", "others", "__weakref__")

    def __init__(self, size, device):
        self.address, self.size, self.device, self.others = 0, size, device, None
        self.stream = _stream_of(device)
        if size:
            self.address = _alloc(size, self.stream)

    def __del__(self):
        if self.address and _free is not None:
            if self.others:
                self._order()
            _free(self.address)

    def record_stream(self, stream):
        """The memory is used on ``stream``: what that holds now comes before its reuse."""
        self.others = (self.others or []) + [stream]

    def _order(self):
        # the allocator hands the memory to later work of the stream it was allocated for
        cuda = _torch.cuda
        mine = (cuda.ExternalStream(self.stream, device=self.device) if self.stream
                else cuda.default_stream(self.device))
        for other in self.others:
            mine.wait_stream(other)

    @property
    def __cuda_array_interface__(self):
        return {"shape": (self.size,), "typestr": "|u1", "data": (self.address, False),
                "version": 2}

    def tensor(self):
        """A uint8 tensor of these bytes, which keeps them."""
        device = f"cuda:{self.device}"
        if not self.size:
            return _torch.empty(0, dtype=_torch.uint8, device=device)
        return _torch.as_tensor(self, device=device)


def _name(table, value, what):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{what} is one of {', '.join(table)}, not {value!r}") from None


class Q8:
    """An 8-bit checkpoint of a ``rows`` x ``cols`` matrix.

    ``codes`` is a (rows, >= cols) and ``scales`` a (rows, >= ceil(cols / 32))
    uint8 CUDA tensor; both start on 16-byte boundaries and have row strides
    that are multiples of 16.  ``format`` is "int8" or "e4m3".
    """

    __slots__ = ("_codes", "_scales", "_memory", "device", "rows", "cols", "format", "struct")

    def __init__(self, codes, scales, cols, format="int8"):
        u8 = (_torch or _load_torch()).uint8
        fmt = _name(Q8_FORMATS, format, "format")
        if (codes.dtype is not u8 or scales.dtype is not u8 or codes.dim() != 2
                or scales.dim() != 2 or not codes.is_cuda):
            raise ValueError("codes and scales must be 2-D uint8 CUDA tensors")
        self.device = device = codes.get_device()
        if scales.get_device() != device:
            raise ValueError("codes and scales must be on one device")
        (rows, width), (rows2, width2) = codes.shape, scales.shape
        blocks = (cols + 31) >> 5
        if cols < 0 or rows2 != rows or width < cols or width2 < blocks:
            raise ValueError("codes must be (rows, >= cols), scales (rows, >= ceil(cols / 32))")
        (ldc, one), (lds, one2) = codes.stride(), scales.stride()
        at, at2 = codes.data_ptr(), scales.data_ptr()
        if rows <= 1:
            ldc, lds = (width + 15) & ~15, (width2 + 15) & ~15
        if rows and cols and (one != 1 or one2 != 1 or (at | at2 | ldc | lds) & 15
                              or ldc < cols or lds < blocks):
            raise ValueError("codes and scales must have contiguous rows, 16-byte aligned bases "
                             "and row strides that are multiples of 16")
        self.struct = Q8Struct(at, at2, ldc, lds, rows, cols, fmt)
        self._codes, self._scales, self._memory = codes, scales, None
        self.rows, self.cols, self.format = rows, cols, format

    @property
    def codes(self):
        """The code bytes, (rows, cols rounded up to 16) for a checkpoint made here."""
        if self._codes is None:
            self._views()
        return self._codes

    @property
    def scales(self):
        """The exponent bytes, one for each block of 32 columns."""
        if self._scales is None:
            self._views()
        return self._scales

    def _views(self):
        s, all_bytes = self.struct, self._memory.tensor()
        at = s.codes - self._memory.address if s.codes else 0
        between, end = at + self.rows * s.ldcodes, at + self.rows * (s.ldcodes + s.ldscales)
        self._codes = all_bytes[at:between].view(self.rows, s.ldcodes)
        self._scales = all_bytes[between:end].view(self.rows, s.ldscales)

    @property
    def nbytes(self) -> int:
        """Bytes that the two tensors hold."""
        return self.codes.numel() + self.scales.numel()

    def record_stream(self, stream) -> None:
        """As ``torch.Tensor.record_stream``, for a checkpoint used on another stream."""
        if self._memory is not None:
            self._memory.record_stream(stream)
        else:
            self._codes.record_stream(stream)
            self._scales.record_stream(stream)

    def __repr__(self):
        return f"Q8({self.rows} x {self.cols}, {self.format})"


def _place(memory, at, device, rows, cols, format, fmt) -> Q8:
    """An uninitialised checkpoint in a piece of memory: codes, then exponents."""
    q = Q8.__new__(Q8)
    ldc, lds = (cols + 15) & ~15, (((cols + 31) >> 5) + 15) & ~15
    base = memory.address + at
    q.struct = Q8Struct(base, base + rows * ldc, ldc, lds, rows, cols, fmt)
    q._codes = q._scales = None
    q._memory = memory
    q.device = device
    q.rows = rows
    q.cols = cols
    q.format = format
    return q


def _bytes(rows, cols) -> int:
    return rows * (((cols + 15) & ~15) + ((((cols + 31) >> 5) + 15) & ~15))


def _make(device, rows, cols, format, fmt) -> Q8:
    return _place(_Memory(_bytes(rows, cols), device), 0, device, rows, cols, format, fmt)


def _make_two(device, rows, cols, format, fmt):
    """Two checkpoints of one shape, kept for one backward pass, in one allocation."""
    one = _bytes(rows, cols)
    memory = _Memory(2 * one, device)
    return (_place(memory, 0, device, rows, cols, format, fmt),
            _place(memory, one, device, rows, cols, format, fmt))


def _matrix(t, what):
    """(rows, cols, row stride) of a float32 CUDA matrix with contiguous rows."""
    if t.dtype is not _torch.float32 or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D float32 CUDA tensor")
    return _strides(t, what)


def _strides(t, what):
    rows, cols = t.shape
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
    fmt = _name(Q8_FORMATS, format, "format")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("a checkpoint is made on a CUDA device")
    with torch.cuda.device(device):
        return _make(torch.cuda.current_device(), rows, cols, format, fmt)


def q8_store(x, format="int8", out=None, stream=None) -> Q8:
    """The 8-bit checkpoint of ``x`` (rows, cols), in ``out`` if given."""
    if _torch is None:
        _load_torch()
    rows, cols, ld = _matrix(x, "x")
    fmt = _name(Q8_FORMATS, format, "format")
    device = x.get_device()
    if stream is not None or _away(device):
        return _elsewhere(lambda: q8_store(x, format, out), device, stream, (x, out))
    q = _make(device, rows, cols, format, fmt) if out is None else _given(out, rows, cols, format,
                                                                     device, "out")
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
    latter splits the tokens into (0: chosen by size).
    """
    if _torch is None:
        _load_torch()
    rows, N, ldy = _matrix(dy, "dy")
    if rows != q.rows:
        raise ValueError(f"dy must have {q.rows} rows, not {rows}")
    code = _name(Q8_ALGOS, algo, "algo")
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
    """``h = act(gate) * up`` and the checkpoints of gate and up: ``(h, gate_q, up_q)``."""
    if _torch is None:
        _load_torch()
    rows, cols, ldg = _matrix(gate, "gate")
    code = _name(ACTS, act, "act")
    fmt = _name(Q8_FORMATS, format, "format")
    device = gate.get_device()
    ldu = _like(up, rows, cols, device, "up")
    if stream is not None or _away(device):
        return _elsewhere(lambda: q8_gated(gate, up, act, format, out, gate_q, up_q), device,
                          stream, (gate, up, out, gate_q, up_q))
    if out is None:
        h, ldh = _empty(rows, cols, 0, device), cols or 1
    else:
        h, ldh = out, _like(out, rows, cols, device, "out")
    if gate_q is None and up_q is None:
        gq, uq = _make_two(device, rows, cols, format, fmt)
    else:
        gq = _make(device, rows, cols, format, fmt) if gate_q is None else _given(
            gate_q, rows, cols, format, device, "gate_q")
        uq = _make(device, rows, cols, format, fmt) if up_q is None else _given(
            up_q, rows, cols, format, device, "up_q")
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
    rows, cols, format, device = gate_q.rows, gate_q.cols, gate_q.format, gate_q.device
    code = _name(ACTS, act, "act")
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
        h_q = _make(device, rows, cols, format, gate_q.struct.format)
    st = _lib.gemm_f32_q8_gated_backward(code, gate_q.struct, up_q.struct, dh.data_ptr(), ldh,
                                         dg.data_ptr(), ldg, du.data_ptr(), ldu,
                                         None if h_q is None else h_q.struct,
                                         _stream_of(device))
    if st:
        _g.check(st, "q8_gated_backward")
    return dg, du, h_q
