"""Matrices whose sizes do not fit 32 bits, on the GPU: refused, with nothing written."""

import pytest

import dense_fp32_gemm_row_gb300 as g

pytestmark = pytest.mark.gpu


def test_a_matrix_wider_than_32_bits():
    import torch

    wide = 2 ** 32 + 8
    q = g.q8_store(torch.ones(1, 1, device="cuda"))
    row = torch.empty((1, wide), device="cuda")
    with pytest.raises(ValueError, match=r"2\^31"):
        g.q8_wgrad(q, row)
    with pytest.raises(ValueError, match=r"2\^31"):
        g.q8_store(row)
    column = row.view(wide, 1)
    with pytest.raises(ValueError, match=r"2\^31"):
        g.q8_store(column)
    codes = torch.zeros((wide, 16), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((wide, 16), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match=r"2\^31"):
        g.Q8(codes, scales, 1)
    fits = g.Q8(codes[:70], scales[:70], 1)
    assert bool((g.q8_restore(fits) == 0).all())
