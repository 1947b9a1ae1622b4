"""The 8-bit integer layers without a GPU: what the library and the binding refuse, and what is a
no-op."""

import ctypes

import pytest

import dense_fp32_gemm_row_gb300 as g
from dense_fp32_gemm_row_gb300 import build as gbuild
from dense_fp32_gemm_row_gb300 import q8
from tests.test_q8_binding import Memory

X, Y, Z, W = 0x7000_0000_0000, 0x7100_0000_0000, 0x7200_0000_0000, 0x7300_0000_0000
BAD = g.ERR_INVALID_VALUE
WIDE = 2 ** 32 + 8  # as an int of 32 bits: 8


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return g.load()


def i8(rows=4, cols=40, codes=X, scales=Y, ld=48):
    return g.I8Struct(codes, scales, ld, rows, cols)


def norm(q, x=Z, ldx=40, r=Z + 0x10000, ldr=40, w=W, eps=1e-6, type=0, s=Z + 0x20000, lds=40):
    return g.gemm_f32_i8_norm(x, ldx, r, ldr, w, eps, type, s, lds, q)


def accepted():
    """What a call that passes its argument checks answers without a GPU."""
    try:
        import torch
        gpu = torch.cuda.is_available()
    except Exception:
        gpu = False
    if gpu:
        pytest.skip("these addresses are no memory: the accepted calls would run on a GPU")
    return g.ERR_UNSUPPORTED_DEVICE


def test_empty_matrices_are_no_ops_without_a_device():
    for q in (i8(rows=0, codes=0, scales=0), i8(cols=0, codes=0, scales=0)):
        assert g.gemm_f32_i8_store(0, 0, 0, q) == g.SUCCESS
        assert norm(q, 0, 0, 0, 0, 0, s=0) == g.SUCCESS
    a, b, none = i8(), i8(rows=7), i8(rows=0, codes=0, scales=0)
    for x, w in ((none, b), (a, none)):
        assert g.gemm_f32_i8_matmul(x, w, 0, 0, 0) == g.SUCCESS
        assert g.gemm_f32_i8_gated(0, x, w, w, 0, 0, 0) == g.SUCCESS


@pytest.mark.parametrize("q", [
    None, i8(rows=-1), i8(cols=-1), i8(codes=0), i8(scales=0), i8(codes=X + 8), i8(scales=Y + 2),
    i8(ld=32), i8(ld=40), i8(ld=0), i8(rows=2 ** 31 - 1, ld=1 << 60)])
def test_bad_matrices_of_codes_are_invalid(q):
    good = i8(rows=9, codes=W, scales=W + 0x10000)
    assert g.gemm_f32_i8_store(Z, 0, 700, q) == BAD
    assert norm(q, ldx=700, ldr=700, lds=700) == BAD
    assert g.gemm_f32_i8_matmul(q, good, Z, 0, 9) == BAD
    assert g.gemm_f32_i8_matmul(good, q, Z, 0, 2 ** 31) == BAD
    for trio in ((q, good, good), (good, q, good), (good, good, q)):
        assert g.gemm_f32_i8_gated(0, *trio, Z, 0, 2 ** 31) == BAD


def test_bad_arguments_are_invalid():
    q, w = i8(), i8(rows=7, codes=W, scales=W + 0x10000)
    for type in (-1, 2, 3):
        assert g.gemm_f32_i8_store(Z, type, 40, q) == BAD
        assert norm(q, type=type) == BAD
        assert g.gemm_f32_i8_gated(0, q, w, w, Z, type, 7) == BAD
    assert g.gemm_f32_i8_matmul(q, w, Z, 3, 7) == BAD
    for x, ld in ((0, 40), (Z + 2, 40), (Z, 39)):
        assert g.gemm_f32_i8_store(x, 0, ld, q) == BAD
        assert norm(q, x=x, ldx=ld) == BAD
        assert norm(q, s=x or Z + 2, lds=ld) == BAD
    assert g.gemm_f32_i8_store(Z + 1, 1, 40, q) == BAD
    assert norm(q, r=Z + 0x10000, ldr=39) == BAD
    assert norm(q, w=0) == BAD and norm(q, w=W + 2) == BAD
    assert norm(q, r=0) == BAD  # a sum without its second term
    for eps in (0.0, -1e-6, 1e-31, float("inf"), float("nan")):
        assert norm(q, eps=eps) == BAD
    for y, ld in ((0, 7), (Z + 2, 7), (Z, 6)):
        assert g.gemm_f32_i8_matmul(q, w, y, 0, ld) == BAD
        assert g.gemm_f32_i8_gated(0, q, w, w, y, 0, ld) == BAD
    for act in (-1, 2):
        assert g.gemm_f32_i8_gated(act, q, w, w, Z, 0, 7) == BAD
    for algo, splits in ((-1, 0), (1, 0), (5, 0), (9, 0), (0, -1), (7, 257)):
        assert g.gemm_f32_i8_matmul(q, w, Z, 0, 7, algo, splits) == BAD
        assert g.gemm_f32_i8_gated(0, q, w, w, Z, 0, 7, algo, splits) == BAD
    # operands of one product have as many columns, those of a gated block one shape
    assert g.gemm_f32_i8_matmul(q, i8(cols=39, codes=W, scales=W + 0x10000), Z, 0, 4) == BAD
    assert g.gemm_f32_i8_gated(0, q, w, i8(rows=8, codes=W, scales=W + 0x10000), Z, 0, 7) == BAD
    # sums that may not fit 32 bits
    for cols, want in ((131072, BAD), (131071, None)):
        a = i8(cols=cols, ld=131072)
        b = i8(rows=7, cols=cols, codes=W, scales=W + 0x1000000, ld=131072)
        if want is None:
            want = accepted()
        assert g.gemm_f32_i8_matmul(a, b, Z, 2, 7) == want
        assert g.gemm_f32_i8_gated(0, a, b, b, Z, 0, 7) == want


def test_the_most_rows():
    most, far = 2 ** 31 - 1024, 0x1000_0000_0000  # far from an output of 4 TB
    for rows, other, want in ((most, 4, None), (most + 1, 4, BAD), (2 ** 31 - 1, 4, BAD),
                              (10 ** 6, 10 ** 6, None), (10 ** 6, 10 ** 6 + 1, BAD)):
        a = i8(rows=rows, cols=16, ld=16)
        b = i8(rows=other, cols=16, codes=W, scales=W + 0x10_0000_0000, ld=16)
        if want is None:
            want = accepted()
        assert g.gemm_f32_i8_matmul(a, b, far, 0, other) == want
        assert g.gemm_f32_i8_matmul(b, a, far, 0, rows) == want
        assert g.gemm_f32_i8_gated(0, a, b, b, far, 1, other) == want
        assert g.gemm_f32_i8_gated(0, b, a, a, far, 1, rows) == want


def test_outputs_apart_from_inputs_and_each_other():
    want = accepted()
    q, w = i8(), i8(rows=7, codes=W, scales=W + 0x10000)
    u = i8(rows=7, codes=W + 0x20000, scales=W + 0x30000)
    assert g.gemm_f32_i8_store(Z, 0, 40, q) == want
    assert g.gemm_f32_i8_store(X - 160, 0, 40, q) == BAD
    assert g.gemm_f32_i8_store(Y + 8, 0, 40, q) == BAD
    assert norm(q) == want and norm(q, s=0) == want and norm(q, r=0, s=0) == want
    assert norm(q, s=Z) == BAD and norm(q, s=Z + 0x10000) == BAD and norm(q, w=Z + 0x20004) == BAD
    assert norm(q, s=X) == BAD and norm(q, x=Y) == BAD
    # the sum beside its terms in one buffer's rows, and one column too close
    assert norm(q, x=Z, ldx=80, r=Z + 0x10000, ldr=80, s=Z + 160, lds=80) == want
    assert norm(q, x=Z, ldx=80, r=Z + 0x10000, ldr=80, s=Z + 156, lds=80) == BAD
    assert g.gemm_f32_i8_matmul(q, w, Z, 0, 7) == want
    assert g.gemm_f32_i8_matmul(q, q, Z, 0, 4) == want  # inputs may be one matrix
    assert g.gemm_f32_i8_gated(0, q, w, u, Z, 0, 7) == want
    for y in (X + 16, Y, W, W + 0x10000 - 4):
        assert g.gemm_f32_i8_matmul(q, w, y, 0, 7) == BAD
        assert g.gemm_f32_i8_gated(0, q, w, u, y, 0, 7) == BAD
    for y in (W + 0x20000, W + 0x30000):
        assert g.gemm_f32_i8_gated(0, q, w, u, y, 0, 7) == BAD


def test_struct_and_constants_match_the_header(tmp_path):
    import os
    import subprocess

    src = tmp_path / "layout.c"
    fields = [n for n, _ in g.I8Struct._fields_]
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n"
                   "typedef void* cudaStream_t; typedef void* cudaEvent_t;\n"
                   "#include \"gemm_f32.h\"\nint main(void){\n"
                   + "".join(f'printf("%zu ", offsetof(gemm_f32_i8, {f}));' for f in fields)
                   + 'printf("%zu %d %d %d %d %d %d\\n", sizeof(gemm_f32_i8), GEMM_F32_TYPE_F32, '
                   "GEMM_F32_TYPE_BF16, GEMM_F32_TYPE_I32, GEMM_F32_I8_MAX_COLS, "
                   "GEMM_F32_I8_STREAM_ROWS, "
                   "GEMM_F32_I8_LEAST_EPS == 1e-30f); return 0; }\n")
    (tmp_path / "cuda_runtime_api.h").write_text("")
    exe = tmp_path / "layout"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", str(tmp_path), "-I", os.path.join(root, "include"), str(src),
                    "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [getattr(g.I8Struct, f).offset for f in fields] + [
        ctypes.sizeof(g.I8Struct), g.TYPE_F32, g.TYPE_BF16, g.TYPE_I32, g.I8_MAX_COLS, g.I8_STREAM_ROWS, 1]


# ---- the binding, on stand-ins for CUDA tensors ---------------------------------------------------

torch = pytest.importorskip("torch")


class Vector(Memory):
    def dim(self):
        return 1

    def stride(self):
        return (1,)

    def numel(self):
        return self.shape[0]


def floats(rows, cols, dtype=torch.float32, device=0):
    return Memory((rows, cols), dtype, device)


def matrix(rows, cols, device=0):
    return g.I8(Memory((rows, -(-cols // 16) * 16), torch.int8, device),
                Vector((rows,), torch.float32, device), cols)


@pytest.fixture(scope="module", autouse=True)
def loaded(lib):
    q8._load_torch()


def weight(cols, dtype=torch.float32, device=0):
    return Vector((cols,), dtype, device)


def calls(x, q, **more):
    return (lambda: g.i8_store(x, **more), lambda: g.i8_norm(x, weight(x.shape[1]), **more),
            lambda: g.i8_matmul(q, q, **more), lambda: g.i8_gated(q, q, q, **more))


def test_a_stream_of_another_device():
    class Stream:
        device = torch.device("cuda", 1)

    for call in calls(floats(8, 64), matrix(8, 64), stream=Stream):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_operands_of_another_device():
    x, q, other = floats(8, 64), matrix(8, 64), matrix(8, 64, device=1)
    for call in (lambda: g.i8_store(x, out=other), lambda: g.i8_norm(x, weight(64), out=other),
                 lambda: g.i8_norm(x, weight(64, device=1)),
                 lambda: g.i8_norm(x, weight(64), residual=floats(8, 64, device=1)),
                 lambda: g.i8_matmul(q, other), lambda: g.i8_gated(q, q, other),
                 lambda: g.I8(q.codes, other.scales, 64),
                 lambda: g.i8_matmul(q, q, out=floats(8, 8, device=1))):
        with pytest.raises(ValueError, match="one device"):
            call()


@pytest.mark.parametrize("size", [2 ** 31, WIDE])
def test_sizes_beyond_32_bits(size):
    q = matrix(1, 1)
    for call in (lambda: g.i8_store(floats(size, 1)), lambda: g.i8_store(floats(1, size)),
                 lambda: g.i8_norm(floats(1, size), weight(size)),
                 lambda: g.i8_matmul(q, q, out=floats(size, 1)), lambda: matrix(size, 1),
                 lambda: matrix(1, size), lambda: g.i8_empty(size, 1), lambda: g.i8_empty(1, size),
                 lambda: g.I8Struct(0, 0, 16, size, 1), lambda: g.I8Struct(0, 0, 16, 1, size)):
        with pytest.raises(ValueError, match=r"2\^31"):
            call()
    assert matrix(2 ** 31 - 1, 1).struct.rows == 2 ** 31 - 1


def test_types_and_shapes():
    x, h, q, w = floats(8, 64), floats(8, 64, torch.float16), matrix(8, 64), weight(64)
    total = floats(8, 64)
    for call in (lambda: g.i8_store(h), lambda: g.i8_norm(h, w), lambda: g.i8_matmul(q, q, dtype=torch.float16),
                 lambda: g.i8_gated(q, q, q, dtype=torch.int32), lambda: g.i8_gated(q, q, q, act="relu"),
                 lambda: g.i8_norm(x, weight(63)), lambda: g.i8_norm(x, weight(64, torch.bfloat16)),
                 lambda: g.i8_norm(x, w, residual=floats(8, 63)), lambda: g.i8_norm(x, w, total=total),
                 lambda: g.i8_norm(x, w, residual=floats(8, 64, torch.bfloat16)),
                 lambda: g.i8_norm(x, w, eps=0.0), lambda: g.i8_norm(x, w, eps=float("nan")),
                 lambda: g.i8_store(x, out=matrix(8, 63)), lambda: g.i8_matmul(q, matrix(8, 63)),
                 lambda: g.i8_gated(q, q, matrix(9, 64)), lambda: g.i8_matmul(q, q, out=floats(8, 9)),
                 lambda: g.i8_matmul(q, q, dtype=torch.bfloat16, out=floats(8, 8)),
                 lambda: g.i8_matmul(q, q, algo="ffma"), lambda: g.i8_gated(q, q, q, algo="ffma"),
                 lambda: g.i8_matmul(q, q, algo="single", splits=2 ** 32 + 1),
                 lambda: g.i8_matmul(matrix(1, 131072), matrix(1, 131072)),
                 lambda: g.I8(q.codes, q.scales, 65), lambda: g.I8(q.codes, weight(9), 64),
                 lambda: g.I8(q.codes, weight(8, torch.float64), 64), lambda: g.I8(x, q.scales, 64),
                 lambda: g.I8(Memory((8, 40), torch.int8), q.scales, 40),  # rows 40 bytes apart
                 lambda: g.i8_empty(-1, 4), lambda: g.i8_empty(4, 4, device="cpu"),
                 lambda: g.i8_store(torch.zeros(4, 40)),
                 lambda: g.I8(torch.zeros(4, 48, dtype=torch.int8), torch.zeros(4), 40)):
        with pytest.raises(ValueError):
            call()


def test_memory_that_is_gone():
    q = matrix(8, 64)
    q.codes.nbytes = lambda: 8 * 64 - 1
    with pytest.raises(ValueError, match="memory"):
        q.struct
    with pytest.raises(ValueError, match="memory"):
        g.i8_matmul(q, q, out=floats(8, 8))
