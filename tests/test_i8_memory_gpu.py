"""8-bit integer layers on matrices whose memory ends with their last column."""

import numpy as np
import pytest

import dense_fp32_gemm_row_gb300 as g
from tests import _i8
from tests.test_i8_gpu import dtype, quiet, sums_of, t, up

pytestmark = pytest.mark.gpu


def ending(rows, cols, gap=0):
    """An I8 whose two tensors' storages hold not a byte behind its last element."""
    torch = t()
    ld = (cols + 15) // 16 * 16 + 16 * gap
    codes = torch.full(((rows - 1) * ld + cols,), 77, dtype=torch.int8, device="cuda")
    q = g.I8(codes.as_strided((rows, cols), (ld, 1)), torch.empty(rows, device="cuda"), cols)
    assert q.codes.untyped_storage().nbytes() == (rows - 1) * ld + cols
    return q


def random_ending(rng, rows, cols, gap=0):
    torch = t()
    q = ending(rows, cols, gap)
    codes = rng.integers(-128, 128, (rows, cols)).astype(np.int8)
    q.codes.copy_(torch.from_numpy(codes))
    q.scales.fill_(1e-3)
    return q, codes


@pytest.mark.parametrize("module", [True, False])
@pytest.mark.parametrize("N,K", [(1, 1), (33, 15), (16, 17), (130, 40), (64, 65), (100, 1025), (257, 4099), (300, 8191)])
@pytest.mark.parametrize("T", [1, 5, 9, 20, 32, 50, 200])
def test_products(T, N, K, module, monkeypatch):
    import dense_fp32_gemm_row_gb300.i8 as binding

    torch = t()
    rng = np.random.default_rng(T * 31 + N * 7 + K)
    (qa, a), (qb, b), (qc, _) = (random_ending(rng, rows, K, gap) for rows, gap in ((T, 0), (N, 1), (N, 0)))
    if not module:
        monkeypatch.setattr(binding, "_native", None)
    want = torch.from_numpy(sums_of(a, b)).to(torch.int32)
    forms = ["auto", "pair", "single"] + ["stream"] * (T <= g.I8_STREAM_ROWS)
    for algo in forms:
        assert torch.equal(g.i8_matmul(qa, qb, dtype=torch.int32, algo=algo).cpu(), want)
    gated = [g.i8_gated(qa, qb, qc, algo=algo) for algo in forms]
    assert all(torch.equal(h, gated[0]) for h in gated)
    quiet()


@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 17), (40, 1000), (2, 4099), (1, 20001)])
def test_rows(rows, cols, name):
    torch = t()
    rng = np.random.default_rng(rows + cols)
    x = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).to(dtype(name)).cuda()
    codes, scales = _i8.store(x.float().cpu().numpy())
    q = ending(rows, cols)
    g.i8_store(x, out=q)
    assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), scales)
    w = up(np.ones((1, cols), np.float32), name)[0]
    g.i8_norm(x, w, out=q)
    assert np.array_equal(q.codes.cpu().numpy(), codes)  # the norm's factor is the scale's alone
    quiet()
