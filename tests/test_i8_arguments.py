"""Arguments that the 8-bit integer layers' binding refuses, without a GPU, and alike with and
without its module on one."""

import pytest

import dense_fp32_gemm_row_gb300 as g
from tests.test_i8_abi import floats, lib, loaded, weight  # noqa: F401

torch = pytest.importorskip("torch")

LARGEST = 2.0 ** 128 - 2.0 ** 104                # of float32
BAD_EPS = (0.0, -1e-6, 9.99999e-31, 2.0 ** 128 - 2.0 ** 103, 1e39, float("inf"), float("nan"))


@pytest.mark.parametrize("eps", BAD_EPS)
def test_eps(eps):
    with pytest.raises(ValueError, match="eps"):
        g.i8_norm(floats(8, 64), weight(64), eps=eps)


@pytest.mark.gpu
@pytest.mark.parametrize("module", [True, False])
def test_eps_with_and_without_the_module(module, monkeypatch):
    import dense_fp32_gemm_row_gb300.i8 as binding

    x, w = torch.randn(3, 40, device="cuda"), torch.ones(40, device="cuda")
    g.i8_norm(x, w)
    assert binding._native is not None
    if not module:
        monkeypatch.setattr(binding, "_native", None)
    for eps in BAD_EPS:
        with pytest.raises(ValueError, match="eps"):
            g.i8_norm(x, w, eps=eps)
    # the least and the largest, which is rounded down to a float; a whole number
    for eps in (1e-30, LARGEST, 2.0 ** 128 - 2.0 ** 103 - 2.0 ** 80, 1):
        q, _ = g.i8_norm(x, w, eps=eps)
        assert bool(torch.isfinite(q.scales).all())


def test_raw_arguments_beyond_32_bits():
    """Whose low 32 bits would be arguments as they should be: before any look at device or memory."""
    q = g.I8Struct(0x7000_0000_0000, 0x7100_0000_0000, 48, 4, 40)
    w = g.I8Struct(0x7200_0000_0000, 0x7300_0000_0000, 48, 7, 40)
    y, wide = 0x7400_0000_0000, 2 ** 32
    assert g.gemm_f32_i8_store(y, wide, 40, q) == g.ERR_INVALID_VALUE
    assert g.gemm_f32_i8_norm(y, 40, 0, 0, y + 0x10000, 1e-6, wide + 1, 0, 0, q) == g.ERR_INVALID_VALUE
    for type, algo, splits in ((wide, 0, 0), (0, wide, 0), (0, wide + 7, 0), (0, 7, wide + 2), (0, 7, -wide),
                               (-wide, 0, 0)):
        assert g.gemm_f32_i8_matmul(q, w, y, type, 7, algo, splits) == g.ERR_INVALID_VALUE
        assert g.gemm_f32_i8_gated(0, q, w, w, y, type, 7, algo, splits) == g.ERR_INVALID_VALUE
    assert g.gemm_f32_i8_gated(wide, q, w, w, y, 0, 7) == g.ERR_INVALID_VALUE


def test_more_tokens_than_the_streaming_kernel_takes():
    """Refused whatever else there is to do, and without a device."""
    y = 0x7400_0000_0000
    for K, N in ((40, 7), (0, 7), (40, 0)):
        a = g.I8Struct(0x7000_0000_0000, 0x7100_0000_0000, 48, g.I8_STREAM_ROWS + 1, K)
        b = g.I8Struct(0x7200_0000_0000, 0x7300_0000_0000, 48, N, K)
        assert g.gemm_f32_i8_matmul(a, b, y, 0, 7, g.ALGO_I8_STREAM) == g.ERR_INVALID_VALUE
        assert g.gemm_f32_i8_gated(0, a, b, b, y, 0, 7, g.ALGO_I8_STREAM) == g.ERR_INVALID_VALUE
