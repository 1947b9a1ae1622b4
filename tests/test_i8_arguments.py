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
