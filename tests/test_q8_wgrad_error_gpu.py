"""How far the tensor-core weight gradient is from its 64-bit value, and alpha and beta in the kernel
itself.

The error of a sum.  Products are exact.  A unit of up to 512 tokens is summed 128 tokens at a time,
a longer one 256: in 24 or 48 additions (three a 16 tokens), each of which may truncate the running sum
to 24 bits.  That loses half a unit in the last place on average: 2^-24 of the sum's binade, 2^-24 *
0.721 = 4.3e-8 of the sum itself (the mean of 1 / m over mantissas m spread evenly in their logarithm).

2-norm.  With terms of random signs the sum of the running sums S_k, k = 1 .. n, has the size n S_n /
sqrt 3, so n truncations make 4.3e-8 * n / sqrt 3: 6.0e-7 for 24, 1.19e-6 for 48.  What single
truncations differ from their mean (0.29 units in the last place) adds 4.3e-8 * 0.58 * sqrt(n / 2) =
8.6e-8 or 1.2e-7, and adding up to 256 such sums in fp32, each rounded by 2^-24 / sqrt 3 at most, of a
total that grows alike, up to 2^-24 / sqrt 3 * sqrt(256 / 2) = 3.9e-7: for the 32 here 1.4e-7.  Squares
added: 6.3e-7 and 1.21e-6.

Each element.  A truncation loses less than 2^-23 of a sum that is at most the chunk's sum |x^| |dY|: 24
or 48 times 2^-23 of sum |x^| |dY| altogether, and 2^-24 of it for each chunk that is added.
"""

import numpy as np
import pytest

import dense_fp32_gemm_row_gb300 as g
from tests import _q8

pytestmark = pytest.mark.gpu

SHORT, LONG = (24, 6.5e-7), (48, 1.25e-6)  # additions a sum, 2-norm over 2-norm
FORMS = ("3xbf16_pair", "3xbf16_single")


def t():
    import torch
    return torch


@pytest.fixture(autouse=True)
def no_device_fault():
    yield
    t().cuda.synchronize()
    g.check(g.gemm_f32_device_status(1), "device status")


def device(a):
    return t().from_numpy(np.ascontiguousarray(a)).cuda()


def case(seed, T, D, N, fmt):
    """A checkpoint, its values in 64 bits, and dY."""
    rng = np.random.default_rng(seed)
    q = g.q8_store(device(_q8.activations(rng, T, D)), format=fmt)
    dy = (1e-3 * rng.standard_normal((T, N)) * np.exp(rng.standard_normal((T, 1)))).astype(np.float32)
    return q, g.q8_restore(q).double().cpu().numpy(), dy


def check(got, x, dy, bounds, alpha=1.0, beta=0.0, old=None):
    additions, norm = bounds
    dy = dy.astype(np.float64)
    product = alpha * (x.T @ dy)
    size = abs(alpha) * (np.abs(x).T @ np.abs(dy))
    kept = beta * old.astype(np.float64) if beta else np.zeros_like(product)
    err = np.abs(got.double().cpu().numpy() - (product + kept))
    # the product with alpha and the fused addition round once each
    last = 2.0 ** -24 * (np.abs(product) + np.abs(product + kept)) if (alpha, beta) != (1.0, 0.0) else 0.0
    assert np.all(err <= (additions * 2.0 ** -23 + (1 + x.shape[0] / 128) * 2.0 ** -24) * size + last)
    assert np.linalg.norm(err) <= norm * np.linalg.norm(product) + np.linalg.norm(last)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt", _q8.FORMATS)
@pytest.mark.parametrize("T,splits,bounds", [
    (128, 1, SHORT), (250, 1, SHORT), (512, 1, SHORT), (513, 1, LONG), (1024, 1, LONG),
    (1024, 2, SHORT), (4096, 1, LONG), (4096, 8, SHORT), (4096, 4, LONG)])
def test_error_of_a_sum(form, fmt, T, splits, bounds):
    q, x, dy = case(T, T, 300, 300, fmt)
    check(g.q8_wgrad(q, device(dy), algo=form, splits=splits), x, dy, bounds)


@pytest.mark.parametrize("T,D,N", [(64, 512, 512), (1000, 1025, 1023), (2048, 512, 512)])
def test_error_where_the_library_chooses(T, D, N):
    """Sizes whose units have no more than 512 tokens, whole or shared."""
    q, x, dy = case(T, T, D, N, "int8")
    check(g.q8_wgrad(q, device(dy)), x, dy, SHORT)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("fmt", _q8.FORMATS)
@pytest.mark.parametrize("T,D,N", [(33, 40, 50), (500, 260, 300), (1000, 513, 260)])
@pytest.mark.parametrize("alpha,beta", [(0.5, 0.0), (1.0, 1.0), (-2.0, 0.25), (1.0, -1.0)])
@pytest.mark.parametrize("splits", [1, 3])
def test_alpha_and_beta_in_the_kernel_and_in_the_sum(form, fmt, T, D, N, alpha, beta, splits):
    """One range of tokens: the kernel itself scales and adds; three: the second kernel does."""
    torch = t()
    q, x, dy = case(T, T, D, N, fmt)
    old = (1e-2 * np.random.default_rng(9).standard_normal((D, N))).astype(np.float32)
    buf = torch.full((D, N + 3), float("nan"), device="cuda")
    out = buf[:, :N]
    if beta:  # else what was there is not read: it stays NaN
        out.copy_(device(old))
    assert g.q8_wgrad(q, device(dy), out=out, alpha=alpha, beta=beta, algo=form, splits=splits) is out
    check(out, x, dy, SHORT if T <= 512 * splits else LONG, alpha, beta, old)
    assert bool(torch.isnan(buf[:, N:]).all())


@pytest.mark.parametrize("form", FORMS + ("ffma",))
def test_accumulation_over_micro_batches(form):
    """beta = 1, as a training step adds its micro-batches, against the batch as a whole."""
    q, x, dy = case(3, 900, 300, 260, "int8")
    dw = None
    for i in range(3):
        part = slice(300 * i, 300 * i + 300)
        qi = g.q8_store(device(x[part].astype(np.float32)))
        assert np.array_equal(g.q8_restore(qi).double().cpu().numpy(), x[part])
        dw = g.q8_wgrad(qi, device(dy[part]), out=dw, beta=0.0 if dw is None else 1.0, algo=form)
    # three sums of at most 256 fp32 additions or 24 truncations, and two additions of them
    check(dw, x, dy, (256 / 2, SHORT[1] + 2.0 ** -23))


@pytest.mark.parametrize("form", FORMS + ("ffma",))
@pytest.mark.parametrize("fmt", _q8.FORMATS)
def test_gradients_near_the_least_floats(form, fmt):
    """dY of 2^-110 and more enters exactly.  Below, its three parts hold it down to the least bf16
    number, 2^-133: on the tensor core it is cut to a multiple of that; on the CUDA cores it is exact."""
    T, D, N = 16, 32, 512
    x = np.zeros((T, D), dtype=np.float32)
    x[np.arange(T), np.arange(T)] = 2.0 ** 100  # so that what enters is seen in dW, which is normal
    q = g.q8_store(device(x), format=fmt)
    rng = np.random.default_rng(0)
    for e in (-100, -109, -110, -111, -114, -118, -122, -126, -127, -131, -134, -149):
        y = (rng.uniform(1, 2, (T, N)) * rng.choice([-1.0, 1.0], (T, N)) * 2.0 ** e).astype(np.float32)
        enters = y.astype(np.float64)
        if form != "ffma":
            enters = np.trunc(enters * 2.0 ** 133) * 2.0 ** -133
            assert e < -110 or np.array_equal(enters, y)
        want = np.zeros((D, N))
        want[:T] = enters * 2.0 ** 100
        assert np.array_equal(g.q8_wgrad(q, device(y), algo=form).double().cpu().numpy(), want)


def test_e4m3_beyond_its_largest_float():
    """248 * 2^120 and more rounds to 2^128: an infinity, which gradients do not hide."""
    torch = t()
    x = torch.ones(4, 64, device="cuda")
    x[1, 3], x[2, 40] = 3.2e38, 3.4e38  # 248 * 2^120 is 3.2964e38
    q = g.q8_store(x, format="e4m3")
    for dtype in (torch.float32, torch.bfloat16):
        back = g.q8_restore(q, dtype=dtype).float()
        assert float(back[1, 3]) == 240 * 2.0 ** 120 and float(back[2, 40]) == float("inf")
    dw = g.q8_wgrad(q, torch.ones(4, 8, device="cuda"))
    assert not torch.isfinite(dw[40]).any() and torch.isfinite(dw[:3]).all()
    assert torch.isfinite(g.q8_restore(g.q8_store(x))).all()  # int8 takes the nearest value it has
