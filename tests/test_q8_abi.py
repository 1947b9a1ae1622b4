"""The 8-bit checkpoint entry points without a GPU: what they refuse, what is
a no-op, and the 64-bit forms that the GPU tests compare with."""

import ctypes

import numpy as np
import pytest

import dense_fp32_gemm_row_gb300 as g
from dense_fp32_gemm_row_gb300 import build as gbuild
from tests import _q8

X, Y, Z, W = 0x7000_0000_0000, 0x7100_0000_0000, 0x7200_0000_0000, 0x7300_0000_0000
BAD = g.ERR_INVALID_VALUE


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return g.load()


def q8(rows=4, cols=40, fmt=0, codes=X, scales=Y, ldc=48, lds=16):
    return g.Q8Struct(codes, scales, ldc, lds, rows, cols, fmt)


def test_empty_matrices_are_no_ops_without_a_device():
    for q in (q8(rows=0, codes=0, scales=0), q8(cols=0, codes=0, scales=0)):
        assert g.gemm_f32_q8_store(0, 0, q) == g.SUCCESS
        assert g.gemm_f32_q8_restore(q, 0, 0) == g.SUCCESS
        assert g.gemm_f32_q8_gated(0, 0, 0, 0, 0, 0, 0, q, q) == g.SUCCESS
        assert g.gemm_f32_q8_gated_backward(0, q, q, 0, 0, 0, 0, 0, 0, q) == g.SUCCESS
    assert g.gemm_f32_q8_wgrad(q8(), 0, 0, 0, 1.0, 0.0, 0, 0) == g.SUCCESS
    assert g.gemm_f32_q8_wgrad(q8(cols=0), 0, 0, 5, 1.0, 0.0, 0, 0) == g.SUCCESS


@pytest.mark.parametrize("q", [
    None, q8(rows=-1), q8(cols=-1), q8(fmt=2), q8(fmt=-1), q8(codes=0), q8(scales=0),
    q8(codes=X + 8), q8(scales=Y + 4), q8(ldc=32), q8(ldc=40), q8(lds=8), q8(lds=0),
    q8(cols=600, ldc=608, lds=16), q8(rows=2 ** 31 - 1, ldc=1 << 60)])
def test_bad_checkpoints_are_invalid(q):
    f = 4 * 700
    assert g.gemm_f32_q8_store(Z, 700, q) == BAD
    assert g.gemm_f32_q8_restore(q, Z, 700) == BAD
    assert g.gemm_f32_q8_wgrad(q, Z, 5, 5, 1.0, 0.0, W, 5) == BAD
    good = q8(codes=W, scales=W + 0x10000)
    assert g.gemm_f32_q8_gated(0, Z, 700, Z + 1000 * f, 700, Z + 2000 * f, 700, good, q) == BAD
    assert g.gemm_f32_q8_gated(0, Z, 700, Z + 1000 * f, 700, Z + 2000 * f, 700, q, good) == BAD
    assert g.gemm_f32_q8_gated_backward(0, good, q, Z, 700, Z + 1000 * f, 700, Z + 2000 * f,
                                        700) == BAD


def test_bad_matrices_are_invalid():
    q = q8()
    assert g.gemm_f32_q8_store(0, 40, q) == BAD
    assert g.gemm_f32_q8_store(Z + 2, 40, q) == BAD
    assert g.gemm_f32_q8_store(Z, 39, q) == BAD
    assert g.gemm_f32_q8_restore(q, 0, 40) == BAD
    assert g.gemm_f32_q8_restore(q, Z + 2, 40) == BAD
    assert g.gemm_f32_q8_restore(q, Z + 1, 40, g.Q8_TO_BF16) == BAD
    assert g.gemm_f32_q8_restore(q, Z, 40, 2) == BAD
    assert g.gemm_f32_q8_wgrad(q, Z, 5, -1, 1.0, 0.0, W, 5) == BAD
    assert g.gemm_f32_q8_wgrad(q, Z, 4, 5, 1.0, 0.0, W, 5) == BAD
    assert g.gemm_f32_q8_wgrad(q, Z, 5, 5, 1.0, 0.0, W, 4) == BAD
    assert g.gemm_f32_q8_wgrad(q, 0, 5, 5, 1.0, 0.0, W, 5) == BAD
    assert g.gemm_f32_q8_wgrad(q, Z, 5, 5, 1.0, 0.0, 0, 5) == BAD
    assert g.gemm_f32_q8_wgrad(q, Z + 2, 5, 5, 1.0, 0.0, W, 5) == BAD
    u = q8(codes=W, scales=W + 0x10000)
    for act in (-1, 2):
        assert g.gemm_f32_q8_gated(act, Z, 40, Z + 0x1000, 40, Z + 0x2000, 40, q, u) == BAD
        assert g.gemm_f32_q8_gated_backward(act, q, u, Z, 40, Z + 0x1000, 40, Z + 0x2000,
                                            40) == BAD
    # two checkpoints of one unit have one shape and format
    for other in (q8(rows=3, codes=W, scales=W + 0x10000), q8(cols=39, codes=W, scales=W + 0x10000),
                  q8(fmt=1, codes=W, scales=W + 0x10000)):
        assert g.gemm_f32_q8_gated(0, Z, 40, Z + 0x1000, 40, Z + 0x2000, 40, q, other) == BAD
        assert g.gemm_f32_q8_gated_backward(0, q, other, Z, 40, Z + 0x1000, 40, Z + 0x2000,
                                            40) == BAD
        assert g.gemm_f32_q8_gated_backward(0, q, u, Z, 40, Z + 0x1000, 40, Z + 0x2000, 40,
                                            other) == BAD


def _no_device_status():
    # what a call that passes its argument checks answers here
    try:
        import torch
        gpu = torch.cuda.is_available()
    except Exception:
        gpu = False
    return None if gpu else g.ERR_UNSUPPORTED_DEVICE


def test_outputs_apart_from_inputs_and_each_other():
    want = _no_device_status()
    if want is None:
        pytest.skip("these addresses are no memory: the accepted calls would run on a GPU")
    q, u = q8(), q8(codes=W, scales=W + 0x10000)
    # gate and up, and their gradients, as the halves of one buffer's rows
    assert g.gemm_f32_q8_gated(0, Z, 80, Z + 160, 80, Z + 0x10000, 40, q, u) == want
    assert g.gemm_f32_q8_gated_backward(0, q, u, Z + 0x10000, 40, Z, 80, Z + 160, 80) == want
    # the second half first
    assert g.gemm_f32_q8_gated_backward(0, q, u, Z + 0x10000, 40, Z + 160, 80, Z, 80) == want
    # one column too close, from either side
    assert g.gemm_f32_q8_gated_backward(0, q, u, Z + 0x10000, 40, Z, 80, Z + 156, 80) == BAD
    assert g.gemm_f32_q8_gated_backward(0, q, u, Z + 0x10000, 40, Z, 79, Z + 160, 79) == BAD
    # h over gate; dgate over dh; codes within the input
    assert g.gemm_f32_q8_gated(0, Z, 40, Z + 0x10000, 40, Z, 40, q, u) == BAD
    assert g.gemm_f32_q8_gated_backward(0, q, u, Z, 40, Z, 40, Z + 0x10000, 40) == BAD
    assert g.gemm_f32_q8_store(X - 160, 40, q) == BAD
    assert g.gemm_f32_q8_restore(q, X + 16, 40) == BAD
    assert g.gemm_f32_q8_gated(0, Z, 40, Z + 0x10000, 40, Z + 0x20000, 40, q, q) == BAD
    assert g.gemm_f32_q8_gated_backward(0, q, u, Z, 40, Z + 0x10000, 40, Z + 0x20000, 40, u) == BAD
    # the gradient over dY, over the checkpoint
    assert g.gemm_f32_q8_wgrad(q, Z, 5, 5, 1.0, 0.0, Z + 4 * 19, 5) == BAD
    assert g.gemm_f32_q8_wgrad(q, Z, 5, 5, 1.0, 0.0, X, 5) == BAD
    assert g.gemm_f32_q8_wgrad(q, Z, 5, 5, 1.0, 0.0, W, 5) == want


def test_binding_refuses_what_it_cannot_hold():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 40)
    for call in (lambda: g.q8_store(x), lambda: g.Q8(torch.zeros(4, 48, dtype=torch.uint8),
                                                    torch.zeros(4, 16, dtype=torch.uint8), 40),
                 lambda: g.q8_gated(x, x)):
        with pytest.raises(ValueError):
            call()


def test_struct_matches_the_header(tmp_path):
    # sizes and offsets as the C compiler lays them out
    import os
    import subprocess

    src = tmp_path / "layout.c"
    fields = [n for n, _ in g.Q8Struct._fields_]
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n"
                   "typedef void* cudaStream_t; typedef void* cudaEvent_t;\n"
                   "#include \"gemm_f32.h\"\nint main(void){\n"
                   + "".join(f'printf("%zu ", offsetof(gemm_f32_q8, {f}));' for f in fields)
                   + 'printf("%zu\\n", sizeof(gemm_f32_q8)); return 0; }\n')
    (tmp_path / "cuda_runtime_api.h").write_text("")
    exe = tmp_path / "layout"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", str(tmp_path), "-I", os.path.join(root, "include"), str(src),
                    "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [getattr(g.Q8Struct, f).offset for f in fields] + [ctypes.sizeof(g.Q8Struct)]


# ---- the 64-bit forms themselves ----------------------------------------------------------------


@pytest.mark.parametrize("fmt,most", [("int8", 127.0), ("e4m3", 448.0)])
def test_reference_scale_is_the_smallest_that_fits(fmt, most):
    rng = np.random.default_rng(1)
    x = _q8.activations(rng, 50, 100)
    codes, e = _q8.store(x, fmt)
    scale = np.exp2(e.astype(np.float64) - (133 if fmt == "int8" else 127))
    xb = np.zeros((50, 4 * 32))
    xb[:, :100] = np.abs(x)
    top = xb.reshape(50, 4, 32).max(axis=2)
    assert np.all(top <= most * scale) and np.all(top > most * scale / 2)
    # no code nearer to the value
    v = _q8.values(codes, e, fmt)
    s = np.repeat(scale, 32, axis=1)[:, :100]
    grid = np.arange(-127, 128) if fmt == "int8" else _q8.E4M3[~np.isnan(_q8.E4M3)]
    best = np.abs(x[:, :, None] - grid[None, None, :] * s[:, :, None]).min(axis=2)
    assert np.array_equal(np.abs(x - v), best)


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_reference_slope_against_differences(name):
    z = np.linspace(-12, 12, 481)
    h = 1e-5
    diff = (_q8.act(z + h, name)[0] - _q8.act(z - h, name)[0]) / (2 * h)
    # truncation h^2 / 6 |act'''| (< 2), cancellation 2^-52 |act| / h
    assert np.max(np.abs(_q8.act(z, name)[1] - diff)) < h * h + 2.0 ** -52 * 13 / h
