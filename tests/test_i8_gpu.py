"""The 8-bit integer layers on the GPU against their plain forms."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest

import dense_fp32_gemm_row_gb300 as g
from tests import _i8, _q8

pytestmark = pytest.mark.gpu

TYPES = ("float32", "bfloat16")


def t():
    import torch
    return torch


def dtype(name):
    return getattr(t(), name)


def up(x: np.ndarray, name="float32", pad=0, offset=0):
    """x on the GPU as a matrix of row stride cols + pad, offset elements into its buffer."""
    torch = t()
    rows, cols = x.shape
    buf = torch.full((offset + rows * (cols + pad) + 8,), float("nan"), device="cuda",
                     dtype=dtype(name))
    m = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return m


def down(x) -> np.ndarray:
    return x.float().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def filled(rows, cols, fill=99, gap=0):
    """An I8 whose rows lie in a wider buffer full of `fill`, and what of it is not the matrix's."""
    torch = t()
    ld = (cols + 15) // 16 * 16 + 16 * gap
    codes = torch.full((rows + 2, ld), fill, dtype=torch.int8, device="cuda")
    scales = torch.full((rows + 2,), float(fill), device="cuda")
    q = g.I8(codes[1:rows + 1, :max(cols, 1)] if cols else codes[1:rows + 1], scales[1:rows + 1], cols)

    def untouched():
        rest = codes.clone()
        rest[1:rows + 1, :cols] = fill
        return bool((rest == fill).all()) and bool((scales[[0, -1]] == fill).all())
    return q, untouched


def quiet():
    t().cuda.synchronize()
    g.check(g.gemm_f32_device_status(1), "device status")


def activations(rng, rows, cols, name="float32"):
    x = _q8.activations(rng, rows, cols)
    return down(t().from_numpy(x).to(dtype(name)))  # values of that type


# ---- rows to 8 bits -------------------------------------------------------------------------------

SHAPES = [(1, 1), (1, 7), (3, 8), (2, 31), (5, 256), (9, 257), (1, 1000), (37, 1000), (700, 130),
          (400, 1024), (305, 1025), (2, 4096), (310, 4096), (306, 5001), (1, 8192), (311, 8200), (2, 16384),
          (1, 16385), (3, 20000), (2, 40001)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_store(rows, cols, name):
    rng = np.random.default_rng(rows * 7 + cols)
    x = activations(rng, rows, cols, name)
    want, scales = _i8.store(x)
    for pad, offset in ((0, 0), (8, 8), (1, 0), (3, 5)):
        q, untouched = filled(rows, cols, gap=pad % 2)
        assert g.i8_store(up(x, name, pad, offset), out=q) is q
        quiet()
        assert np.array_equal(down(q.codes)[:, :cols], want)
        assert np.array_equal(down(q.scales), scales)
        assert untouched()
    q = g.i8_store(up(x, name))
    assert np.array_equal(down(q.codes)[:, :cols], want) and (q.rows, q.cols) == (rows, cols)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm(rows, cols, residual, name):
    torch = t()
    rng = np.random.default_rng(rows * 11 + cols)
    x = activations(rng, rows, cols, name)
    r = activations(rng, rows, cols, name) if residual else None
    w = down(torch.from_numpy((1 + 0.3 * rng.standard_normal(cols)).astype(np.float32)).to(dtype(name)))
    eps = 1e-5
    codes, scales, s = _i8.norm(x, r, w, eps)
    wt = up(w[None], name)[0]
    for pad, offset in ((0, 0), (8, 8), (3, 5)):
        q, untouched = filled(rows, cols)
        total = up(np.zeros_like(x), name, pad, offset) if residual else None
        got, sums = g.i8_norm(up(x, name, pad, offset), wt,
                              residual=up(r, name, pad, offset) if residual else None, eps=eps,
                              out=q, total=total)
        quiet()
        assert got is q and sums is total and untouched()
        assert np.array_equal(down(q.codes)[:, :cols], codes)
        assert np.max(np.abs(down(q.scales) / scales - 1)) < _i8.norm_bound(cols)
        if residual:
            assert torch.equal(sums.cpu(), torch.from_numpy(s).to(dtype(name)))


def test_norm_of_weights_off_a_boundary():
    rng = np.random.default_rng(4)
    x, w = activations(rng, 5, 300), (1 + rng.standard_normal(300)).astype(np.float32)
    codes, scales, _ = _i8.norm(x, None, w, 1e-6)
    q, s = g.i8_norm(up(x), up(w[None], offset=1)[0])
    assert s is None and np.array_equal(down(q.codes)[:, :300], codes)
    assert np.max(np.abs(down(q.scales) / scales - 1)) < _i8.norm_bound(300)


@pytest.mark.parametrize("cols", [5, 300, 9000, 20000])
def test_rows_of_special_values(cols):
    torch = t()
    top = np.float32(3.4e38)
    x = np.zeros((10, cols), np.float32)
    x[1, -1] = np.nan
    x[2, 0] = np.inf
    x[3, 2] = -np.inf
    x[4] = 1e-40                        # below 2^-100: subnormal
    x[5] = 2.0 ** -100
    x[6] = np.where(np.arange(cols) % 2, top, -top)
    x[7] = 1.5
    x[8, 1] = -0.0
    x[9, cols // 2] = -2.0 ** -90
    want, scales = _i8.store(x)
    q = g.i8_store(up(x))
    quiet()
    assert np.array_equal(down(q.codes)[:, :cols], want)
    assert np.array_equal(down(q.scales), scales, equal_nan=True)
    assert np.isnan(down(q.scales)[1:4]).all() and (down(q.codes)[1:4, :cols] == 0).all()
    # squares of row 6 are beyond fp32, its norm is not
    w = np.full(cols, 0.5, np.float32)
    codes, scales, _ = _i8.norm(x, None, w, 1e-6)
    q, _ = g.i8_norm(up(x), up(w[None])[0])
    quiet()
    got = down(q.scales)
    assert np.array_equal(down(q.codes)[:, :cols], codes)
    assert np.isnan(got[1:4]).all()
    fine = np.array([6, 7])
    assert np.max(np.abs(got[fine] / scales[fine] - 1)) < _i8.norm_bound(cols)
    # magnitudes below 2^-100 count as that in the scale: codes are as many steps of it
    assert np.allclose(got[[0, 4, 5, 8]], 2.0 ** -100 / 127 / 1e-3, rtol=1e-5)
    # a sum that only the residual makes infinite
    big = up(np.full((2, cols), 3e38, np.float32))
    q, s = g.i8_norm(big, up(w[None])[0], residual=big)
    assert torch.isinf(s).all() and torch.isnan(q.scales).all() and (q.codes[:, :cols] == 0).all()


def test_least_eps():
    x = np.full((1, 64), 1e-14, np.float32)
    w = np.ones(64, np.float32)
    codes, scales, _ = _i8.norm(x, None, w, 1e-30)
    q, _ = g.i8_norm(up(x), up(w[None])[0], eps=1e-30)
    assert np.array_equal(down(q.codes)[:, :64], codes)
    assert abs(down(q.scales)[0] / scales[0] - 1) < _i8.norm_bound(64)


def test_squares_and_eps_beyond_float32_together():
    x = np.full((3, 40), 1.8e19, np.float32)  # squares of 3.24e38, a mean below the largest float
    x[1, 1:] = 0
    x[2] = 1
    w = np.linspace(0.5, 2, 40, dtype=np.float32)
    codes, scales, _ = _i8.norm(x, None, w, float(np.float32(3e38)))
    q, _ = g.i8_norm(up(x), up(w[None])[0], eps=3e38)
    assert np.array_equal(down(q.codes)[:, :40], codes)
    assert (np.abs(down(q.scales) / scales - 1) < _i8.norm_bound(40)).all()


# ---- products -------------------------------------------------------------------------------------


def operand(rng, rows, cols, most=127, gap=0):
    """An I8 of random codes between padding that must not be read, its codes and scales."""
    torch = t()
    q, _ = filled(rows, cols, fill=77, gap=gap)
    codes = rng.integers(-most - 1, most + 1, (rows, cols)).astype(np.int8)
    scales = np.exp(rng.standard_normal(rows) - 4).astype(np.float32)
    if cols:
        q.codes[:, :cols].copy_(torch.from_numpy(codes))
    q.scales.copy_(torch.from_numpy(scales))
    return q, codes, scales


def sums_of(a, b):
    torch = t()
    return (torch.from_numpy(a).cuda().double() @ torch.from_numpy(b).cuda().double().t()).cpu().numpy()


def output(rows, cols, name, pad=0, offset=0):
    """An output with guards around it, and whether they are as they were."""
    torch = t()
    ld = cols + pad
    buf = torch.full((offset + rows * ld + 64,), 55, device="cuda", dtype=dtype(name))
    y = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]

    def untouched():
        rest = buf.clone()
        rest[offset:offset + rows * ld].view(rows, ld)[:, :cols] = 55
        return bool((rest == 55).all())
    return y, untouched


PRODUCTS = [(1, 1, 1), (1, 5, 3), (2, 16, 16), (1, 130, 1000), (1, 512, 2048), (3, 1000, 65),
            (7, 33, 129), (8, 64, 64), (9, 257, 1024), (15, 1023, 300), (16, 128, 1025), (17, 300, 2047),
            (24, 2048, 1024), (31, 31, 31), (32, 640, 512), (33, 129, 128), (47, 200, 4100), (48, 96, 256),
            (64, 128, 64), (65, 127, 63), (100, 1000, 77), (127, 129, 127), (128, 128, 128), (129, 257, 191),
            (200, 40, 5000), (255, 256, 1023), (256, 256, 256), (257, 513, 320), (300, 1000, 1025),
            (512, 512, 2049), (1000, 1023, 1025), (1025, 300, 448), (70, 3, 9000), (2000, 17, 33),
            (640, 1280, 512), (1, 4097, 4096), (5, 8, 131071), (300, 20, 65540)]


@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_matmul(T, N, K):
    rng = np.random.default_rng(T * 31 + N * 7 + K)
    qa, a, sa = operand(rng, T, K, gap=T % 2)
    qb, b, sb = operand(rng, N, K, gap=N % 2)
    acc = sums_of(a, b)
    y, untouched = output(T, N, "int32", pad=N % 3, offset=T % 2)
    assert g.i8_matmul(qa, qb, out=y) is y
    quiet()
    assert np.array_equal(down(y), acc.astype(np.int64)) and untouched()
    want = acc * sa.astype(np.float64)[:, None] * sb.astype(np.float64)
    for name in TYPES:
        y, untouched = output(T, N, name, pad=T % 4, offset=N % 5)
        g.i8_matmul(qa, qb, out=y)
        quiet()
        assert untouched()
        bound = _i8.rounded(_i8.value_bound(want), want, name)
        assert np.all(np.abs(down(y) - want) <= bound)
    assert t().equal(g.i8_matmul(qa, qb, dtype=dtype("bfloat16")), y)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_gated(T, N, K, act, name):
    rng = np.random.default_rng(T * 29 + N * 5 + K)
    qa, a, sa = operand(rng, T, K)
    (qg, b, sb), (qu, c, sc) = operand(rng, N, K, gap=1), operand(rng, N, K)
    # activations' arguments of a few units
    for q, s in ((qg, sb), (qu, sc)):
        s /= 60 * np.sqrt(K)
        q.scales.copy_(t().from_numpy(s))
    y, untouched = output(T, N, name, pad=N % 3, offset=T % 2)
    assert g.i8_gated(qa, qg, qu, act=act, out=y) is y
    quiet()
    assert untouched()
    sa, sb, sc = (s.astype(np.float64) for s in (sa, sb, sc))
    gate, upv = sums_of(a, b) * sa[:, None] * sb, sums_of(a, c) * sa[:, None] * sc
    want = _q8.act(gate, act)[0] * upv
    bound = _i8.rounded(_i8.gated_bound(gate, upv, act), want, name)
    assert np.all(np.abs(down(y) - want) <= bound)


@pytest.mark.parametrize("algo,splits", [("pair", 0), ("single", 1), ("single", 2), ("single", 3), ("single", 5), ("single", 8), ("single", 256), ("stream", 0)])
@pytest.mark.parametrize("T,N,K", PRODUCTS[::3] + [(257, 129, 1024), (513, 1023, 1088), (129, 513, 8200)])
def test_forced_forms(T, N, K, algo, splits):
    torch = t()
    if algo == "stream" and T > g.I8_STREAM_ROWS:
        some = g.i8_empty(T, K)
        with pytest.raises(g.GemmError):
            g.i8_matmul(some, some, algo=algo)
        return
    rng = np.random.default_rng(T + N + K)
    qa, a, _ = operand(rng, T, K)
    (qb, b, sb), (qc, _, sc) = operand(rng, N, K), operand(rng, N, K)
    for q, s in ((qb, sb), (qc, sc)):
        q.scales.copy_(torch.from_numpy(s / 60 / np.sqrt(K).astype(np.float32)))
    y, untouched = output(T, N, "int32", pad=1)
    g.i8_matmul(qa, qb, out=y, algo=algo, splits=splits)
    quiet()
    assert np.array_equal(down(y), sums_of(a, b).astype(np.int64)) and untouched()
    for act in ("silu", "gelu"):
        y, untouched = output(T, N, "float32", pad=1)
        g.i8_gated(qa, qb, qc, act=act, out=y, algo=algo, splits=splits)
        assert torch.equal(y, g.i8_gated(qa, qb, qc, act=act)) and untouched()
    quiet()


@pytest.mark.parametrize("T,N,K", [(1, 40, 131071), (6, 33, 131071), (20, 300, 33000), (300, 300, 5000),
                                   (257, 130, 131071), (70, 4, 20000)])
@pytest.mark.parametrize("a,b", [(-128, -128), (127, -128), (-128, 127)])
def test_sums_of_the_largest_products(T, N, K, a, b):
    """Sums far beyond 2^24, where fp32 no longer holds every integer: odd ones from a last column."""
    torch = t()
    q, w = g.i8_empty(T, K), g.i8_empty(N, K)
    for m, v in ((q, a), (w, b)):
        m.codes.fill_(99)
        m.codes[:, :K] = v
        m.codes[:, K - 1] = 1
    want = a * b * (K - 1) + 1
    assert bool((g.i8_matmul(q, w, dtype=torch.int32) == want).all())
    quiet()


@pytest.mark.parametrize("T", [3, 40, 200])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_of_all_sizes(T, act):
    """One code a row, so that gate and up are what their scales say."""
    torch = t()
    g64 = np.array([0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 5, -5, 13, -13, 20, -20, 60, -60, 86, -86, 87.5, -87.5, 88,
                    -88, 89, -89, 100, -100, 1e4, -1e4, 1e30, -1e30])
    N = len(g64)
    one = g.i8_empty(T, 1)
    one.codes.zero_()
    one.codes[:, 0] = 1
    one.scales.fill_(1.0)
    w, v = g.i8_empty(N, 1), g.i8_empty(N, 1)
    for m, s in ((w, g64), (v, np.full(N, 3.0))):
        m.codes.zero_()
        m.codes[:, 0] = 1
        m.scales.copy_(torch.from_numpy(s.astype(np.float32)))
    gate = np.tile(g64.astype(np.float32).astype(np.float64), (T, 1))
    got = down(g.i8_gated(one, w, v, act=act)).astype(np.float64)
    quiet()
    want = _q8.act(gate, act)[0] * 3.0
    assert np.all(np.abs(got - want) <= _i8.gated_bound(gate, np.full((T, N), 3.0), act))
    w.scales.fill_(float("inf"))
    assert bool((g.i8_gated(one, w, v, act=act) == float("inf")).all())


def test_scales_that_are_no_numbers():
    torch = t()
    rng = np.random.default_rng(8)
    for T in (5, 200):
        qa, a, sa = operand(rng, T, 100)
        qb, b, sb = operand(rng, 70, 100)
        sa[1], sa[2], sb[3] = np.nan, np.inf, np.nan
        a[2] = np.abs(a[2] | 1) & 127
        b[4] = 0
        for q, c, s in ((qa, a, sa), (qb, b, sb)):
            q.codes[:, :100].copy_(torch.from_numpy(c))
            q.scales.copy_(torch.from_numpy(s))
        with np.errstate(invalid="ignore"):
            want = (sums_of(a, b).astype(np.float32) * sa[:, None]) * sb
        got = down(g.i8_matmul(qa, qb))
        assert np.array_equal(got, want, equal_nan=True)
        assert np.isnan(got[1]).all() and np.isnan(got[:, 3]).all() and np.isnan(got[2, 4])
        assert np.isnan(down(g.i8_gated(qa, qb, qb))[1]).all()


@pytest.mark.parametrize("N,K", [(1000, 1025), (640, 4096), (64, 20000)])
def test_a_token_does_not_depend_on_the_others(N, K):
    torch = t()
    rng = np.random.default_rng(N + K)
    qa, _, _ = operand(rng, 700, K)
    (qb, _, sb), (qc, _, sc) = operand(rng, N, K), operand(rng, N, K)
    for q, s in ((qb, sb), (qc, sc)):
        q.scales.copy_(torch.from_numpy(s / 60 / np.sqrt(K).astype(np.float32)))
    whole, gated = g.i8_matmul(qa, qb), g.i8_gated(qa, qb, qc, act="gelu")
    for first, n in ((0, 1), (5, 2), (11, 8), (30, 17), (60, 40), (100, 100), (333, 129), (400, 300)):
        part = g.I8(qa.codes[first:first + n], qa.scales[first:first + n], K)
        assert torch.equal(g.i8_matmul(part, qb), whole[first:first + n])
        assert torch.equal(g.i8_gated(part, qb, qc, act="gelu"), gated[first:first + n])


def test_empty_matrices():
    torch = t()
    none, some, flat = g.i8_empty(0, 64), g.i8_store(torch.ones(5, 64, device="cuda")), g.i8_empty(3, 0)
    assert g.i8_matmul(none, some).shape == (0, 5) and g.i8_matmul(some, none).shape == (5, 0)
    assert g.i8_gated(none, some, some).shape == (0, 5)
    flat.scales.fill_(1.0)
    for name in TYPES + ("int32",):
        y, untouched = output(3, 3, name, pad=2, offset=1)
        assert bool((g.i8_matmul(flat, flat, out=y) == 0).all()) and untouched()
    y, untouched = output(3, 3, "bfloat16", pad=1, offset=1)
    assert bool((g.i8_gated(flat, flat, flat, out=y) == 0).all()) and untouched()
    assert g.i8_store(torch.empty(0, 7, device="cuda")).rows == 0
    assert g.i8_norm(torch.empty(0, 7, device="cuda"), torch.ones(7, device="cuda"))[0].rows == 0


# ---- a block of them, streams, threads and graphs ---------------------------------------------------


class Block:
    """A gated block's operators as they are used."""

    def __init__(self, T, D, F, name, seed=0):
        torch = t()
        rng = np.random.default_rng(seed)
        self.x, self.r = (up(activations(rng, T, D, name), name) for _ in range(2))
        self.w = up((1 + 0.1 * rng.standard_normal((1, D))).astype(np.float32), name)[0]
        self.gate, self.up, self.down = (
            g.i8_store(torch.from_numpy((rng.standard_normal(s) / np.sqrt(s[1])).astype(np.float32)).cuda())
            for s in ((F, D), (F, D), (D, F)))
        self.name = name

    def __call__(self):
        q, s = g.i8_norm(self.x, self.w, residual=self.r)
        h = g.i8_gated(q, self.gate, self.up, dtype=dtype(self.name))
        hq = g.i8_store(h)
        return {"q": q, "s": s, "h": h, "hq": hq, "y": g.i8_matmul(hq, self.down, dtype=dtype(self.name))}


def flat(made):
    return [x for v in made.values() for x in ((v.codes[:, :v.cols], v.scales) if isinstance(v, g.I8) else (v,))]


def same(a, b):
    return all(t().equal(x, y) for x, y in zip(flat(a), flat(b)))


@pytest.mark.parametrize("T,D,F,name", [(1, 256, 640, "bfloat16"), (3, 250, 333, "float32"), (24, 512, 1280, "bfloat16"),
                                        (130, 257, 700, "float32"), (700, 640, 1280, "bfloat16")])
def test_block(T, D, F, name):
    """Each step against its plain form on what the step before gave."""
    b = Block(T, D, F, name, seed=T)
    made = b()
    quiet()
    q, hq = made["q"], made["hq"]
    codes, scales, s = _i8.norm(down(b.x), down(b.r), down(b.w), 1e-6)
    assert np.array_equal(down(q.codes)[:, :D], codes)
    assert np.max(np.abs(down(q.scales) / scales - 1)) < _i8.norm_bound(D)
    assert t().equal(made["s"].cpu(), t().from_numpy(s).to(dtype(name)))

    def product(a, w):
        return sums_of(down(a.codes)[:, :a.cols], down(w.codes)[:, :a.cols]) * \
            down(a.scales).astype(np.float64)[:, None] * down(w.scales).astype(np.float64)
    gate, upv = product(q, b.gate), product(q, b.up)
    want = _q8.act(gate, "silu")[0] * upv
    assert np.all(np.abs(down(made["h"]) - want) <= _i8.rounded(_i8.gated_bound(gate, upv, "silu"), want, name))
    codes, scales = _i8.store(down(made["h"]))
    assert np.array_equal(down(hq.codes)[:, :F], codes) and np.array_equal(down(hq.scales), scales)
    want = product(hq, b.down)
    assert np.all(np.abs(down(made["y"]) - want) <= _i8.rounded(_i8.value_bound(want), want, name))


def test_block_is_near_the_float_block():
    """The whole chain against the block in 64 bits: 8-bit rounding is all that is lost."""
    torch = t()
    T, D, F = 200, 512, 1024
    b = Block(T, D, F, "float32", seed=5)
    y = down(b()["y"]).astype(np.float64)
    s = down(b.x).astype(np.float64) + down(b.r)
    n = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + 1e-6) * down(b.w)

    def weights(w):
        return down(w.codes)[:, :w.cols] * down(w.scales).astype(np.float64)[:, None]
    h = _q8.act(n @ weights(b.gate).T, "silu")[0] * (n @ weights(b.up).T)
    want = h @ weights(b.down).T
    # activations are rounded twice, each time by up to half of a 127th of the row's largest
    # magnitude (uniform, so a step of 1 / sqrt(12)): relative to a row's 2-norm step sqrt(D) / sqrt(12).
    # norm: three products of relative error e1 in h; h: e2 in y; doubled for the spread of rows.
    def relative(z):
        return np.max(np.abs(z).max(axis=1) / 127 * np.sqrt(z.shape[1] / 12) / np.linalg.norm(z, axis=1))
    bound = 2 * (3 * relative(n) + relative(h))
    assert np.linalg.norm(y - want) / np.linalg.norm(want) < bound
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 40])
def test_the_binding_without_its_module(T, monkeypatch):
    """The quick calls and the step by step ones: the same results, of the same kind."""
    import dense_fp32_gemm_row_gb300.i8 as binding

    b = Block(T, 250, 333, "bfloat16")
    want = b()
    assert binding._native is not None
    plain, none = g.i8_norm(b.x, b.w)
    monkeypatch.setattr(binding, "_native", None)
    got = b()
    q, s = g.i8_norm(b.x, b.w)
    quiet()
    assert same(got, want) and none is None and s is None and same({"q": q}, {"q": plain})
    for x, y in zip(flat(got), flat(want)):
        assert x.shape == y.shape and x.stride() == y.stride() and x.dtype == y.dtype
    for x, y in ((got["q"], want["q"]), (got["hq"], want["hq"])):
        assert (x.rows, x.cols, x.device, x.nbytes, x.codes.shape) == (y.rows, y.cols, y.device, y.nbytes, y.codes.shape)


def test_matrices_whose_memory_is_gone():
    torch = t()
    q = g.i8_store(torch.randn(5, 70, device="cuda"))
    w = g.i8_store(torch.randn(9, 70, device="cuda"))
    q.codes.untyped_storage().resize_(0)
    for call in (lambda: g.i8_matmul(q, w), lambda: g.i8_matmul(w, q), lambda: g.i8_gated(q, w, w),
                 lambda: g.i8_store(torch.ones(5, 70, device="cuda"), out=q)):
        with pytest.raises(ValueError, match="memory"):
            call()


@pytest.mark.parametrize("T", [1, 20, 300])
def test_another_stream(T):
    torch = t()
    b = Block(T, 512, 1024, "bfloat16")
    want = b()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        under = b()
    q, s = g.i8_norm(b.x, b.w, residual=b.r, stream=side)
    h = g.i8_gated(q, b.gate, b.up, dtype=torch.bfloat16, stream=side)
    hq = g.i8_store(h, stream=side)
    y = g.i8_matmul(hq, b.down, dtype=torch.bfloat16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    quiet()
    assert same(under, want) and same({"q": q, "s": s, "h": h, "hq": hq, "y": y}, want)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_captured_and_replayed(T):
    torch = t()
    b = Block(T, 512, 1024, "bfloat16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        made = b()
    for seed in (3, 4):
        fresh = Block(T, 512, 1024, "bfloat16", seed=seed)
        b.x.copy_(fresh.x)
        b.r.copy_(fresh.r)
        graph.replay()
        want = b()
        quiet()
        assert same(made, want)


FIRST = """
import torch, dense_fp32_gemm_row_gb300 as g
torch.manual_seed(0)
q = [g.i8_store(torch.randn(r, 4096, device="cuda")) for r in (64, 4096, 4096)]
one = g.i8_matmul(g.i8_store(torch.randn(1, 4096, device="cuda")), q[1])
side = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    y = g.i8_matmul(q[0], q[1], dtype=torch.int32)
    h = g.i8_gated(*q)
graph.replay()
torch.cuda.synchronize()
g.check(g.gemm_f32_device_status(1), "device status")
assert torch.equal(y.double(), q[0].codes.double() @ q[1].codes.double().t())
assert torch.equal(y, g.i8_matmul(q[0], q[1], dtype=torch.int32)) and torch.equal(h, g.i8_gated(*q))
print("captured")
"""


def test_the_first_split_product_is_a_captured_one():
    made = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert made.returncode == 0 and "captured" in made.stdout, made.stderr[-2000:]


def test_graphs_side_by_side():
    """Two graphs of one stream's calls, replayed at the same time as each other and as calls."""
    torch = t()
    blocks = [Block(20, 1024, 4096, "float32", seed=s) for s in range(3)]
    want = [b() for b in blocks]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blocks[0]()
    torch.cuda.current_stream().wait_stream(side)
    graphs, made = [], []
    for b in blocks[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            made.append(b())
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    eager = []
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager.append(blocks[2]())
    quiet()
    assert same(made[0], want[0]) and same(made[1], want[1]) and all(same(e, want[2]) for e in eager)


def test_threads_at_once():
    torch = t()
    blocks = [Block(T, 512, 1024, "bfloat16", seed=T) for T in (1, 7, 40, 300)]
    want = [b() for b in blocks]
    torch.cuda.synchronize()
    made, errors = [[] for _ in blocks], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    made[i].append(blocks[i]())
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(blocks))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    quiet()
    assert not errors
    assert all(same(m, w) for ms, w in zip(made, want) for m in ms)


def test_host_faults():
    """A workspace or a descriptor that cannot be had: reported, nothing written, and gone after."""
    torch = t()
    rng = np.random.default_rng(3)
    qa, a, _ = operand(rng, 40, 4096)
    qb, b, _ = operand(rng, 200, 4096)
    want = sums_of(a, b).astype(np.int64)
    y, _ = output(40, 200, "int32")
    for algo, splits, kind, status in (("single", 16, g.INJECT_WORKSPACE, g.ERR_WORKSPACE),
                                       ("single", 16, g.INJECT_DESCRIPTOR, g.ERR_DESCRIPTOR),
                                       ("pair", 0, g.INJECT_DESCRIPTOR, g.ERR_DESCRIPTOR)):
        g.gemm_f32_release()  # the next split needs its workspace again
        y.fill_(55)
        g.gemm_f32_inject_host_fault(kind)
        try:
            with pytest.raises(g.GemmError) as e:
                g.i8_matmul(qa, qb, out=y, algo=algo, splits=splits)
        finally:
            g.gemm_f32_inject_host_fault(g.INJECT_NONE)
        assert e.value.status == status
        torch.cuda.synchronize()
        assert bool((y == 55).all())
        g.i8_matmul(qa, qb, out=y, algo=algo, splits=splits)
        quiet()
        assert np.array_equal(down(y), want)


def test_weights_side_by_side():
    """Gate and up as the row halves of one matrix, tokens as rows of a larger one."""
    torch = t()
    rng = np.random.default_rng(6)
    for T in (3, 70):
        qa, a, sa = operand(rng, T + 9, 200)
        qw, w, sw = operand(rng, 2 * 150, 200)
        part = g.I8(qa.codes[4:T + 4], qa.scales[4:T + 4], 200)
        gate, upper = (g.I8(qw.codes[i:i + 150], qw.scales[i:i + 150], 200) for i in (0, 150))
        own = [g.i8_empty(m.rows, 200) for m in (part, gate, upper)]
        for m, o in zip((part, gate, upper), own):
            o.codes[:, :200].copy_(m.codes[:, :200])
            o.scales.copy_(m.scales)
        assert torch.equal(g.i8_gated(part, gate, upper), g.i8_gated(*own))
        assert np.array_equal(down(g.i8_matmul(part, upper, dtype=torch.int32)),
                              sums_of(a[4:T + 4], w[150:]).astype(np.int64))


def test_results_do_not_change_from_run_to_run():
    for T in (1, 24, 300):
        b = Block(T, 1024, 2048, "float32")
        first = b()
        assert all(same(b(), first) for _ in range(5))


def test_many_calls_back_to_back():
    """Forms after one another without a wait between, as kernels that start early meet."""
    torch = t()
    rng = np.random.default_rng(12)
    cases = []
    for T, N, K, algo, splits in ((1, 700, 900, "auto", 0), (300, 520, 1100, "pair", 0), (20, 640, 4096, "auto", 0),
                                  (50, 300, 2048, "single", 7), (600, 200, 300, "single", 1), (9, 64, 9000, "single", 2),
                                  (130, 1000, 700, "auto", 0), (257, 129, 2600, "pair", 0)):
        (qa, a, _), (qb, b, _) = operand(rng, T, K), operand(rng, N, K)
        cases.append((qa, qb, algo, splits, torch.from_numpy(sums_of(a, b)).to(torch.int32).cuda()))
    made = [g.i8_matmul(qa, qb, dtype=torch.int32, algo=algo, splits=splits)
            for _ in range(40) for qa, qb, algo, splits, _ in cases]
    quiet()
    for i, y in enumerate(made):
        assert torch.equal(y, cases[i % len(cases)][4])


def test_offsets_beyond_32_bits():
    """Codes, inputs and outputs whose last rows lie beyond 2^31 elements and 2^32 bytes."""
    torch = t()
    rows = 2 ** 21 + 3
    x = torch.zeros((rows, 1040), dtype=torch.bfloat16, device="cuda")
    x[-2, 5], x[-1, 1039] = 2.0, -3.0
    q = g.i8_store(x)
    assert q.codes[-2, 5] == 127 and q.codes[-1, 1039] == -127 and int(q.codes.any(dim=1).sum()) == 2
    total = torch.empty_like(x)
    n, s = g.i8_norm(x, torch.ones(1040, dtype=torch.bfloat16, device="cuda"), residual=x, total=total)
    assert n.codes[-1, 1039] == -127 and s[-1, 1039] == -6.0 and int(s.any(dim=1).sum()) == 2
    del x, total, s, n
    w = g.i8_store(torch.eye(1040, device="cuda"))
    y = g.i8_matmul(q, w, dtype=torch.int32)
    assert y[-1, 1039] == -127 * 127 and y[-2, 5] == 127 * 127 and int(y.any(dim=1).sum()) == 2
    del y
    # the same as weights: output rows beyond 2^32 bytes apart
    few = g.i8_store(torch.eye(1040, device="cuda")[1030:])
    y = g.i8_matmul(few, q, dtype=torch.int32)
    assert y[9, -1] == -127 * 127 and int((y != 0).sum()) == 1
    many = g.I8(w.codes[:700], w.scales[:700], 1040)
    y = g.i8_matmul(many, q, dtype=torch.bfloat16)
    assert y[5, -2] == 2.0 and int((y != 0).sum()) == 1
