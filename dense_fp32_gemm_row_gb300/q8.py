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
    "ACT_SILU", "ACT_GELU", "ACTS", "ALGO_3XBF16", "Q8_ALGOS", "gemm_f32_q8_store", "gemm_f32_q8_restore",
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
Q8_ALGOS = {"auto": 0, "ffma": 1, "3xbf16": ALGO_3XBF16}
ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU}


class Q8Struct(ctypes.Structure):
    """``gemm_f32_q8`` of the C header."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ldcodes", ctypes.c_longlong), ("ldscales", ctypes.c_longlong),
                ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("format", ctypes.c_int)]


# ---- raw entry points: addresses and the stream are plain integers --------------------------


def gemm_f32_q8_store(X, ldx, q, stream=0) -> int:
    return _g.load().gemm_f32_q8_store(_g._p(X), ldx, q, _g._p(stream))


def gemm_f32_q8_restore(q, X, ldx, type=Q8_TO_F32, stream=0) -> int:
    return _g.load().gemm_f32_q8_restore(q, _g._p(X), ldx, type, _g._p(stream))


def gemm_f32_q8_wgrad(x, dY, lddy, N, alpha, beta, dW, lddw, algo=0, splits=0, stream=0) -> int:
    return _g.load().gemm_f32_q8_wgrad(x, _g._p(dY), lddy, N, alpha, beta, _g._p(dW), lddw, algo,
                                       splits, _g._p(stream))


def gemm_f32_q8_gated(act, G, ldg, U, ldu, H, ldh, gq, uq, stream=0) -> int:
    return _g.load().gemm_f32_q8_gated(act, _g._p(G), ldg, _g._p(U), ldu, _g._p(H), ldh, gq, uq,
                                       _g._p(stream))


def gemm_f32_q8_gated_backward(act, gq, uq, dH, lddh, dG, lddg, dU, lddu, hq=None,
                               stream=0) -> int:
    return _g.load().gemm_f32_q8_gated_backward(act, gq, uq, _g._p(dH), lddh, _g._p(dG), lddg,
                                                _g._p(dU), lddu, hq, _g._p(stream))


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


def _name(table, value, what):
    try:
        return table[value]
    except KeyError:
        raise ValueError(f"{what} is one of {', '.join(table)}, not {value!r}") from None


class Q8:
    """An 8-bit checkpoint of a ``rows`` x ``cols`` matrix.

    ``codes`` is a (rows, >= cols) and ``scales`` a (rows, >= ceil(cols / 32))
    uint8 CUDA tensor; both start on 16-byte boundaries and have row strides
    that are multiples of 16.  ``format`` is "int8" or "e4m3".
    """

    __slots__ = ("codes", "scales", "rows", "cols", "format", "struct")

    def __init__(self, codes, scales, cols, format="int8"):
        import torch

        fmt = _name(Q8_FORMATS, format, "format")
        rows, cols = codes.shape[0], int(cols)
        blocks = (cols + Q8_BLOCK - 1) // Q8_BLOCK
        for t, width in ((codes, cols), (scales, blocks)):
            if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_cuda:
                raise ValueError("codes and scales must be 2-D uint8 CUDA tensors")
            if t.shape[0] != rows or t.shape[1] < width:
                raise ValueError("codes must be (rows, >= cols), scales (rows, >= ceil(cols / 32))")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        ldc, lds = _bytes_ld(codes), _bytes_ld(scales)
        self.codes, self.scales = codes, scales
        self.rows, self.cols, self.format = rows, cols, format
        self.struct = Q8Struct(codes.data_ptr(), scales.data_ptr(), ldc, lds, rows, cols, fmt)

    @property
    def nbytes(self) -> int:
        """Bytes that the two tensors hold."""
        return self.codes.numel() + self.scales.numel()

    def __repr__(self):
        return f"Q8({self.rows} x {self.cols}, {self.format})"


def _bytes_ld(t) -> int:
    rows, width = t.shape
    if rows and width and (t.stride(1) != 1 or t.data_ptr() & 15):
        raise ValueError("codes and scales must have contiguous rows and 16-byte aligned bases")
    ld = t.stride(0) if rows > 1 else (width + 15) // 16 * 16
    if ld & 15 or ld < width:
        raise ValueError("row strides of codes and scales must be multiples of 16")
    return ld


def _ld(t, what) -> int:
    """The row stride of a float32 CUDA matrix with contiguous rows."""
    import torch

    if t.dtype != torch.float32 or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D float32 CUDA tensor")
    return _row_stride(t, what)


def _row_stride(t, what) -> int:
    rows, cols = t.shape
    if cols > 1 and rows and t.stride(1) != 1:
        raise ValueError(f"{what} must have contiguous rows")
    if rows <= 1:
        return max(cols, 1)
    ld = t.stride(0)
    if ld < cols:
        raise ValueError(f"{what} must have rows that do not overlap")
    return ld


def _shape(t, shape, what) -> None:
    if tuple(t.shape) != shape:
        raise ValueError(f"{what} must be {shape}, not {tuple(t.shape)}")


class _Call:
    """The device and stream of one call: allocations inside the block belong to the stream."""

    __slots__ = ("device", "stream", "current", "guard", "other")

    def __init__(self, device, stream):
        import torch

        self.device = device
        self.current = torch.cuda.current_stream(device)
        self.other = stream is not None and stream != self.current
        self.stream = stream if self.other else self.current
        self.guard = None

    def __enter__(self):
        import torch

        if self.other:
            self.guard = torch.cuda.stream(self.stream)
        elif self.device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.device)
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False

    def uses(self, *tensors) -> None:
        """Tensors made on the current stream that this call reads or writes on another."""
        if self.other:
            for t in tensors:
                if isinstance(t, Q8):
                    t.codes.record_stream(self.stream)
                    t.scales.record_stream(self.stream)
                elif t is not None:
                    t.record_stream(self.stream)


def _same_device(device, *tensors) -> None:
    for t in tensors:
        if t is not None and (t.codes if isinstance(t, Q8) else t).device != device:
            raise ValueError("all tensors must be on one device")


def q8_empty(rows, cols, format="int8", device="cuda") -> Q8:
    """An uninitialised checkpoint of a rows x cols matrix."""
    import torch

    blocks = (cols + Q8_BLOCK - 1) // Q8_BLOCK
    codes = torch.empty((rows, (cols + 15) // 16 * 16), dtype=torch.uint8, device=device)
    scales = torch.empty((rows, (blocks + 15) // 16 * 16), dtype=torch.uint8, device=device)
    return Q8(codes, scales, cols, format)


def _out_q8(q, rows, cols, format, device, what) -> Q8:
    if q is None:
        return q8_empty(rows, cols, format, device)
    if (q.rows, q.cols) != (rows, cols):
        raise ValueError(f"{what} must hold {rows} x {cols}, not {q.rows} x {q.cols}")
    if q.format != format:
        raise ValueError(f"{what} must be in {format}, not {q.format}")
    return q


def q8_store(x, format="int8", out=None, stream=None) -> Q8:
    """The 8-bit checkpoint of ``x`` (rows, cols), in ``out`` if given."""
    ld = _ld(x, "x")
    _name(Q8_FORMATS, format, "format")
    _same_device(x.device, out)
    with _Call(x.device, stream) as c:
        q = _out_q8(out, x.shape[0], x.shape[1], format, x.device, "out")
        st = gemm_f32_q8_store(x.data_ptr(), ld, q.struct, c.stream.cuda_stream)
        c.uses(x, out)
    _g.check(st, "q8_store")
    return q


def q8_restore(q, out=None, dtype=None, stream=None):
    """The values ``q`` stands for, as float32 or (``dtype=torch.bfloat16``) bfloat16, both exact."""
    import torch

    dtype = dtype or (out.dtype if out is not None else torch.float32)
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dtype is torch.float32 or torch.bfloat16")
    device = q.codes.device
    _same_device(device, out)
    with _Call(device, stream) as c:
        x = torch.empty((q.rows, q.cols), dtype=dtype, device=device) if out is None else out
        if x.dtype != dtype or x.dim() != 2:
            raise ValueError(f"out must be a 2-D {dtype} tensor")
        _shape(x, (q.rows, q.cols), "out")
        st = gemm_f32_q8_restore(q.struct, x.data_ptr(), _row_stride(x, "out"),
                                 Q8_TO_F32 if dtype == torch.float32 else Q8_TO_BF16,
                                 c.stream.cuda_stream)
        c.uses(q, out)
    _g.check(st, "q8_restore")
    return x


def q8_wgrad(q, dy, out=None, alpha=1.0, beta=0.0, algo="auto", splits=0, stream=None):
    """``out = alpha * x_hat.T @ dy + beta * out`` from the checkpoint ``q`` of x.

    ``dy`` is (q.rows, N); ``out`` (q.cols, N) is allocated if not given, and
    must be given for ``beta`` other than 0 (gradient accumulation).  ``algo``
    is "auto", "ffma" or "3xbf16" (the tensor-core kernel), ``splits`` the
    number of ranges the latter splits the tokens into (0: chosen by size).
    """
    import torch

    ldy = _ld(dy, "dy")
    code = _name(Q8_ALGOS, algo, "algo")
    N = dy.shape[1]
    _shape(dy, (q.rows, N), "dy")
    _same_device(q.codes.device, dy, out)
    if out is None and beta != 0.0:
        raise ValueError("beta needs out, the gradient to add to")
    with _Call(dy.device, stream) as c:
        dw = torch.empty((q.cols, N), dtype=torch.float32, device=dy.device) if out is None else out
        _shape(dw, (q.cols, N), "out")
        st = gemm_f32_q8_wgrad(q.struct, dy.data_ptr(), ldy, N, alpha, beta, dw.data_ptr(),
                               _ld(dw, "out"), code, splits, c.stream.cuda_stream)
        c.uses(q, dy, out)
    _g.check(st, "q8_wgrad")
    return dw


def q8_gated(gate, up, act="silu", format="int8", out=None, gate_q=None, up_q=None, stream=None):
    """``h = act(gate) * up`` and the checkpoints of gate and up: ``(h, gate_q, up_q)``."""
    import torch

    ldg, ldu = _ld(gate, "gate"), _ld(up, "up")
    code = _name(ACTS, act, "act")
    _name(Q8_FORMATS, format, "format")
    rows, cols = gate.shape
    _shape(up, (rows, cols), "up")
    device = gate.device
    _same_device(device, up, out, gate_q, up_q)
    with _Call(device, stream) as c:
        h = torch.empty((rows, cols), dtype=torch.float32, device=device) if out is None else out
        _shape(h, (rows, cols), "out")
        gq = _out_q8(gate_q, rows, cols, format, device, "gate_q")
        uq = _out_q8(up_q, rows, cols, format, device, "up_q")
        st = gemm_f32_q8_gated(code, gate.data_ptr(), ldg, up.data_ptr(), ldu, h.data_ptr(),
                               _ld(h, "out"), gq.struct, uq.struct, c.stream.cuda_stream)
        c.uses(gate, up, out, gate_q, up_q)
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
    import torch

    ldh = _ld(dh, "dh")
    code = _name(ACTS, act, "act")
    rows, cols = gate_q.rows, gate_q.cols
    _shape(dh, (rows, cols), "dh")
    if (up_q.rows, up_q.cols, up_q.format) != (rows, cols, gate_q.format):
        raise ValueError("gate_q and up_q must have one shape and one format")
    if h_q is not None and not want_h:
        raise ValueError("h_q given, and want_h false")
    device = dh.device
    _same_device(device, gate_q, up_q, dgate, dup, h_q)
    with _Call(device, stream) as c:
        dg = torch.empty((rows, cols), dtype=torch.float32, device=device) if dgate is None else dgate
        du = torch.empty((rows, cols), dtype=torch.float32, device=device) if dup is None else dup
        _shape(dg, (rows, cols), "dgate")
        _shape(du, (rows, cols), "dup")
        hq = _out_q8(h_q, rows, cols, gate_q.format, device, "h_q") if want_h else None
        st = gemm_f32_q8_gated_backward(code, gate_q.struct, up_q.struct, dh.data_ptr(), ldh,
                                        dg.data_ptr(), _ld(dg, "dgate"), du.data_ptr(),
                                        _ld(du, "dup"), hq.struct if want_h else None,
                                        c.stream.cuda_stream)
        c.uses(gate_q, up_q, dh, dgate, dup, h_q)
    _g.check(st, "q8_gated_backward")
    return dg, du, hq
