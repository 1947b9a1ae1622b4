"""8-bit checkpoint operators on the GPU against their 64-bit forms."""

import gc

import numpy as np
import pytest

import dense_fp32_gemm_row_gb300 as g
from dense_fp32_gemm_row_gb300 import q8 as _binding
from tests import _q8

pytestmark = pytest.mark.gpu

FORMATS = _q8.FORMATS
ACTS = ("silu", "gelu")


def t():
    import torch
    return torch


@pytest.fixture(autouse=True)
def no_device_fault():
    yield
    t().cuda.synchronize()
    g.check(g.gemm_f32_device_status(1), "device status")


def matrix(a, pad=0, offset=0):
    """A device copy of ``a`` whose rows are ``pad`` elements further apart than they are long and
    which starts ``offset`` elements into its buffer (NaN all around), and that buffer."""
    torch = t()
    a = np.ascontiguousarray(a, dtype=np.float32)
    rows, cols = a.shape
    ld = cols + pad
    buf = torch.full((offset + rows * ld + 64,), float("nan"), device="cuda")
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(torch.from_numpy(a))
    return view, buf


def outside_is_nan(view, buf):
    """Whether nothing outside ``view`` was written in its NaN-filled buffer."""
    torch = t()
    view.fill_(float("nan"))
    return bool(torch.isnan(buf).all())


def checkpoint(x, fmt, junk=True):
    """A Q8 of the numpy matrix x made by the 64-bit form, with junk in its padding bytes."""
    torch = t()
    rows, cols = x.shape
    codes, exps = _q8.store(x, fmt)
    nb = exps.shape[1]
    q = g.q8_empty(rows, cols, fmt)
    if junk:
        q.codes.fill_(0x7F)
        q.scales.fill_(0xFF)
    q.codes[:, :cols] = torch.from_numpy(codes).cuda()
    q.scales[:, :nb] = torch.from_numpy(exps).cuda()
    return q, _q8.values(codes, exps, fmt)


def bytes_of(q):
    nb = -(-q.cols // 32)
    return q.codes[:, :q.cols].cpu().numpy(), q.scales[:, :nb].cpu().numpy()


# ---- store and restore ---------------------------------------------------------------------------

SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (3, 127), (5, 128), (7, 129), (2, 1000), (37, 1024),
          (300, 203), (129, 4100), (1, 16385)]
LAYOUTS = [(0, 0), (4, 0), (1, 0), (0, 1), (7, 3)]  # pad, offset


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,offset", LAYOUTS)
def test_store_is_exact(fmt, rows, cols, pad, offset):
    rng = np.random.default_rng(rows * 100003 + cols)
    x = _q8.activations(rng, rows, cols)
    view, _ = matrix(x, pad, offset)
    q = g.q8_empty(rows, cols, fmt)
    q.codes.fill_(0xA5)
    q.scales.fill_(0x5A)
    assert g.q8_store(view, format=fmt, out=q) is q
    codes, exps = bytes_of(q)
    want_codes, want_exps = _q8.store(x, fmt)
    assert np.array_equal(exps, want_exps)
    assert np.array_equal(codes, want_codes)
    # the padding of the rows is the caller's
    assert bool((q.codes[:, cols:] == 0xA5).all())
    assert bool((q.scales[:, -(-cols // 32):] == 0x5A).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_store_at_the_limits_of_the_format(fmt):
    """Blocks of zeros, denormals, the largest floats, and magnitudes at and next to where the
    exponent steps; ties; negative zeros."""
    one = np.float32(1)
    tops = [0.0, 1e-45, 1e-40, 2.0 ** -126, 2.0 ** -120, 3e-36, 3.4028235e38, 3.39e38, 2.0 ** 127]
    for base in (127.0, 448.0, 1.0, 1.984375, 1.75, 63.5, 224.0):
        b = np.float32(base)
        tops += [b, np.nextafter(b, one * 1000), np.nextafter(b, one * 0)]
    rows = []
    for top in tops:
        ramp = np.linspace(-1, 1, 32).astype(np.float64) * float(top)
        ramp[5], ramp[6] = float(top), -0.0
        rows.append(ramp)
        rows.append(np.where(np.arange(32) % 2, 0.5, 1.5) * float(top) / 127 * np.arange(32) / 2)
    x = np.array(rows, dtype=np.float32)
    x = np.where(np.isfinite(x), x, np.float32(3e38))
    for fill in (x, -x, x[:, ::-1].copy()):
        q = g.q8_store(matrix(fill)[0], format=fmt)
        codes, exps = bytes_of(q)
        want_codes, want_exps = _q8.store(fill, fmt)
        assert np.array_equal(exps, want_exps)
        # -0.0: the sign of a zero code is e4m3's alone and restores to a zero
        assert np.array_equal(_q8.values(codes, exps, fmt), _q8.values(want_codes, want_exps, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("cols,pad", [(256, 0), (100, 3)])
def test_a_non_finite_value_takes_its_block(fmt, value, cols, pad):
    x = _q8.activations(np.random.default_rng(3), 9, cols)
    x[2, 40] = x[7, cols - 1] = value
    view, _ = matrix(x, pad)
    q = g.q8_store(view, format=fmt)
    codes, exps = bytes_of(q)
    want_codes, want_exps = _q8.store(x, fmt)
    assert np.array_equal(exps, want_exps) and np.array_equal(codes, want_codes)
    back = g.q8_restore(q).cpu().numpy()
    assert np.isnan(back[2, 32:64]).all() and np.isnan(back[7, cols - 1])
    assert np.array_equal(np.isnan(back), np.isnan(_q8.values(codes, exps, fmt)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,offset", LAYOUTS)
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_restore_is_exact(fmt, rows, cols, pad, offset, kind):
    torch = t()
    dtype = getattr(torch, kind)
    q, want = checkpoint(_q8.activations(np.random.default_rng(cols), rows, cols), fmt)
    ld = cols + pad
    buf = torch.full((offset + rows * ld + 64,), float("nan"), dtype=dtype, device="cuda")
    out = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    assert g.q8_restore(q, out=out) is out
    assert np.array_equal(out.double().cpu().numpy(), want)
    assert outside_is_nan(out, buf)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cols", [256 * 32, 256 * 32 - 5])
def test_restore_of_every_code_and_exponent(fmt, cols):
    """All 256 codes under all 256 exponent bytes, those the store does not write included."""
    torch = t()
    q = g.q8_empty(8, cols, fmt)
    code = np.arange(cols) % 32 + 32 * np.arange(8)[:, None]
    exps = np.tile(np.arange(256), (8, 1)).astype(np.uint8)
    q.codes[:, :cols] = torch.from_numpy(code.astype(np.uint8)).cuda()
    q.scales[:, :256] = torch.from_numpy(exps).cuda()
    want = _q8.values(code.astype(np.uint8), exps, fmt)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)
    for dtype in (torch.float32, torch.bfloat16):
        got = g.q8_restore(q, dtype=dtype).float().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)


# ---- gated units ---------------------------------------------------------------------------------

GATED_SHAPES = [(1, 1), (1, 32), (2, 33), (5, 128), (3, 127), (37, 1000), (64, 1024), (300, 203)]


def halves(a, b, fill=float("nan")):
    """Device views holding a and b side by side in one buffer's rows."""
    torch = t()
    rows, cols = a.shape
    both = torch.full((rows, 2 * cols), fill, device="cuda")
    left, right = both[:, :cols], both[:, cols:]
    if fill != fill:
        left.copy_(torch.from_numpy(a))
        right.copy_(torch.from_numpy(b))
    return left, right


def gate_values(rng, rows, cols):
    z = 2 * rng.standard_normal((rows, cols))
    z.flat[:: 17] *= 8  # both tails
    return z.astype(np.float32)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,cols", GATED_SHAPES)
@pytest.mark.parametrize("side_by_side", [False, True])
def test_gated_forward(fmt, act, rows, cols, side_by_side):
    rng = np.random.default_rng(rows + 7 * cols)
    gate, up = gate_values(rng, rows, cols), _q8.activations(rng, rows, cols)
    dev = halves(gate, up) if side_by_side else (matrix(gate)[0], matrix(up)[0])
    h, gq, uq = g.q8_gated(*dev, act=act, format=fmt)
    for q, x in ((gq, gate), (uq, up)):
        codes, exps = bytes_of(q)
        want_codes, want_exps = _q8.store(x, fmt)
        assert np.array_equal(exps, want_exps) and np.array_equal(codes, want_codes)
    z, u = gate.astype(np.float64), up.astype(np.float64)
    err = np.abs(h.double().cpu().numpy() - _q8.act(z, act)[0] * u)
    assert np.all(err <= (_q8.act_bound(z, act)[0] + 2.0 ** -23 * np.abs(_q8.act(z, act)[0]))
                  * np.abs(u) + 2.0 ** -126)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,cols", GATED_SHAPES)
@pytest.mark.parametrize("side_by_side", [False, True])
def test_gated_backward(fmt, act, rows, cols, side_by_side):
    rng = np.random.default_rng(rows + 11 * cols)
    gq, z = checkpoint(gate_values(rng, rows, cols), fmt)
    uq, u = checkpoint(_q8.activations(rng, rows, cols), fmt)
    dh = (1e-3 * rng.standard_normal((rows, cols))).astype(np.float32)
    dev_dh, _ = matrix(dh)
    dg, du = halves(dh, dh) if side_by_side else (None, None)
    dgate, dup, hq = g.q8_gated_backward(gq, uq, dev_dh, act=act, dgate=dg, dup=du)
    a, slope = _q8.act(z, act)
    ea, es = _q8.act_bound(z, act)
    r = 2.0 ** -23  # the products' own roundings
    d = dh.astype(np.float64)
    assert np.all(np.abs(dgate.double().cpu().numpy() - d * u * slope)
                  <= np.abs(d * u) * (es + 2 * r * np.abs(slope)) + 2.0 ** -126)
    assert np.all(np.abs(dup.double().cpu().numpy() - d * a)
                  <= np.abs(d) * (ea + 2 * r * np.abs(a)) + 2.0 ** -126)
    # h recomputed in 8 bits: within half a step of its exact value, the step being the one of the
    # exponent byte written (for e4m3 an eighth of the value, or the format's least step)
    codes, exps = bytes_of(hq)
    v = _q8.values(codes, exps, fmt)
    scale = np.repeat(np.exp2(exps.astype(np.float64) - (133 if fmt == "int8" else 127)), 32,
                      axis=1)[:, :cols]
    h = a * u
    step = scale if fmt == "int8" else np.maximum(
        np.exp2(np.floor(np.log2(np.maximum(np.abs(h), 1e-300))) - 3), scale * 2.0 ** -9)
    slack = (ea + r * np.abs(a)) * np.abs(u) + 2.0 ** -126
    assert np.all(np.abs(v - h) <= step / 2 * (1 + 1e-5) + slack)
    # and the exponent is the smallest that fits, up to h's own rounding
    top = np.zeros((rows, -(-cols // 32) * 32))
    top[:, :cols] = np.abs(h)
    top = top.reshape(rows, -1, 32).max(axis=2)
    most = (127.0 if fmt == "int8" else 448.0) * np.exp2(
        exps.astype(np.float64) - (133 if fmt == "int8" else 127))
    assert np.all(top <= most * (1 + 1e-4))
    floor = exps == (7 if fmt == "int8" else 10)
    assert np.all((top >= most / 2 * (1 - 1e-4)) | floor)


@pytest.mark.parametrize("act", ACTS)
def test_gated_gradients_against_differences_of_the_forward(act):
    """dgate and dup against central differences of q8_gated, at values the format holds exactly."""
    torch = t()
    rng = np.random.default_rng(5)
    gq, z = checkpoint(gate_values(rng, 40, 96), "int8")
    uq, u = checkpoint(_q8.activations(rng, 40, 96), "int8")
    dh = torch.ones(40, 96, device="cuda")
    dgate, dup, _ = g.q8_gated_backward(gq, uq, dh, act=act, want_h=False)
    zt, ut = torch.from_numpy(z).float().cuda(), torch.from_numpy(u).float().cuda()
    step = 2.0 ** -6

    def forward(a, b):
        return g.q8_gated(a, b, act=act)[0].double()

    by_gate = (forward(zt + step, ut) - forward(zt - step, ut)) / (2 * step)
    by_up = (forward(zt, ut + step) - forward(zt, ut - step)) / (2 * step)
    # truncation step^2 / 6 |act'''| (act''' < 2), rounding of the forward 2^-19 |h| / step and of
    # the shifted arguments (2^-24 |z| |act'|, 2^-24 |u|) / step
    size = (1 + zt.abs()).double()
    rough = step * step / 3 + 2.0 ** -19 * size / step
    assert bool(((dgate.double() - by_gate).abs() <= rough * ut.abs().double()
                 + 2.0 ** -19 * 1e-3).all())
    assert bool(((dup.double() - by_up).abs() <= 2.0 ** -18 * size * (1 + ut.abs().double())
                 / step).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cols", [128, 45])
def test_gated_keeps_a_non_finite_value_in_sight(fmt, cols):
    x = np.ones((3, cols), dtype=np.float32)
    x[1, 33] = np.inf
    h, gq, uq = g.q8_gated(matrix(x)[0], matrix(np.ones_like(x))[0], act="silu", format=fmt)
    assert not np.isfinite(h.cpu().numpy()[1, 33]) and np.isfinite(h.cpu().numpy()[0]).all()
    dgate, dup, hq = g.q8_gated_backward(gq, uq, matrix(np.ones_like(x))[0])
    for out in (dgate, dup, g.q8_restore(hq)):
        out = out.cpu().numpy()
        assert np.isnan(out[1, 32:min(cols, 64)]).all()
        assert np.isfinite(out[1, :32]).all() and np.isfinite(out[0]).all()


# ---- weight gradient -----------------------------------------------------------------------------

# Error of a sum over tokens in fp32, against S = sum |x^| |dY|.  The products are exact; what is
# rounded or truncated is the running sum: by at most 2^-23 of its size at each of at most 32
# additions a 128-token chunk on the tensor core, or 2^-24 at each of 256 on the CUDA cores, and
# 2^-24 at each chunk added after that.  (A worst case: single errors add up like a random walk.)
EACH = 256 * 2.0 ** -24

# The error as a whole, 2-norm over 2-norm.  Truncation by half a unit in the last place on
# average (2^-24 * 0.72 of the sum, relative) at each of 48 additions of a 256-token chunk, with
# the sum two thirds of its final size on average, is 1.4e-6; fp32 additions of the chunks and of
# the CUDA-core sums add less than 4e-7 up to 2^16 tokens.
NORM = 2e-6


def wgrad_case(rng, T, D, N, fmt):
    q, x = checkpoint(_q8.activations(rng, T, D), fmt)
    dy = (1e-3 * rng.standard_normal((T, N)) * np.exp(rng.standard_normal((T, 1)))).astype(np.float32)
    return q, x, dy


def assert_wgrad(got, x, dy, alpha=1.0, beta=0.0, old=None):
    want = alpha * (x.T @ dy.astype(np.float64))
    size = abs(alpha) * (np.abs(x).T @ np.abs(dy.astype(np.float64)))
    chunks = 2 + x.shape[0] / 128
    if old is not None:
        want = want + beta * old.astype(np.float64)
        size = size + np.abs(beta * old)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= (EACH + chunks * 2.0 ** -24) * size + 1e-37)
    norm = np.linalg.norm(want)
    if norm and old is None and want.size >= 16:
        assert np.linalg.norm(err) <= NORM * norm


WGRAD_SHAPES = [(1, 1, 1), (1, 40, 5), (2, 32, 4), (15, 33, 3), (16, 64, 64), (17, 65, 130),
                (31, 127, 129), (32, 128, 256), (33, 257, 255), (63, 100, 200), (64, 256, 256),
                (65, 31, 300), (127, 300, 31), (128, 129, 260), (129, 512, 128), (200, 513, 260),
                (255, 260, 4), (256, 4, 260), (257, 300, 516), (1000, 333, 77), (1025, 1000, 24)]


ALGOS = ("ffma", "3xbf16_pair", "3xbf16_single")
TENSOR = ALGOS[1:]


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("T", [33, 700])
def test_wgrad_of_exact_sums_is_exact(T, algo):
    """Small integers: every product and partial sum fits fp32, so every path gives the same bits."""
    rng = np.random.default_rng(T)
    x = rng.integers(-127, 128, (T, 200)).astype(np.float32)
    x[:, ::32] = 127  # exponent byte 133: the codes are the integers
    dy = rng.integers(-64, 65, (T, 130)).astype(np.float32) + 0.0
    q = g.q8_store(matrix(x)[0])
    assert np.array_equal(g.q8_wgrad(q, matrix(dy)[0], algo=algo).double().cpu().numpy(),
                          x.astype(np.float64).T @ dy.astype(np.float64))


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,D,N", WGRAD_SHAPES)
def test_wgrad(fmt, T, D, N, algo):
    q, x, dy = wgrad_case(np.random.default_rng(T + D + N), T, D, N, fmt)
    assert_wgrad(g.q8_wgrad(q, matrix(dy)[0], algo=algo), x, dy)


@pytest.mark.parametrize("algo", TENSOR)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,D,N,splits", [(100, 40, 50, 1), (100, 40, 50, 2), (100, 40, 50, 4),
                                          (100, 40, 50, 256), (1000, 300, 301, 7),
                                          (5000, 257, 100, 33), (5000, 257, 100, 256)])
def test_wgrad_split_over_tokens(fmt, T, D, N, splits, algo):
    q, x, dy = wgrad_case(np.random.default_rng(T + splits), T, D, N, fmt)
    assert_wgrad(g.q8_wgrad(q, matrix(dy)[0], algo=algo, splits=splits), x, dy)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_wgrad_of_every_code_and_exponent(fmt, algo):
    """All codes the format has under exponents over its whole range, one token at a time in effect
    (dY a one-hot row), so that every output is one exact value."""
    torch = t()
    least = 7 if fmt == "int8" else 10
    exps = np.concatenate([np.arange(least, 248, 12), [least, 133, 127, 247]]).astype(np.uint8)
    code = np.array([c for c in range(256) if fmt == "int8" or c & 127 != 127], dtype=np.uint8)
    code = np.resize(code, 256)
    T, D = len(exps), 256
    q = g.q8_empty(T, D, fmt)
    q.codes[:, :D] = torch.from_numpy(np.tile(code, (T, 1))).cuda()
    q.scales[:, :8] = torch.from_numpy(np.tile(exps[:, None], (1, 8))).cuda()
    got = g.q8_wgrad(q, torch.eye(T, device="cuda"), algo=algo).cpu().numpy()
    want = _q8.values(np.tile(code, (T, 1)), np.tile(exps[:, None], (1, 8)), fmt).T
    # 448 * 2^120 is beyond fp32: an infinity, which times the other columns' zeros is NaN
    over = np.abs(want).max(axis=1) > np.finfo(np.float32).max
    assert over.any() == (fmt == "e4m3")
    assert np.array_equal(got[~over], want[~over].astype(np.float32))
    assert not np.isfinite(got[over]).any()


@pytest.mark.parametrize("algo", ("auto",) + TENSOR)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,D,N", [(4096, 256, 256), (5000, 300, 500), (20000, 256, 40),
                                   (65536, 64, 96), (2048, 2048, 1024), (600, 4100, 1500),
                                   # tiles of 256 x 256 shared by the 76 CTA pairs: 45 and, after
                                   # a round of whole tiles, 14 of 90, over tile boundaries or not
                                   (2100, 1283, 2049), (2100, 2305, 2303)])
def test_wgrad_large(fmt, T, D, N, algo):
    q, x, dy = wgrad_case(np.random.default_rng(T + D + N), T, D, N, fmt)
    assert_wgrad(g.q8_wgrad(q, matrix(dy)[0], algo=algo), x, dy)


@pytest.mark.parametrize("algo", ("auto",) + TENSOR)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,D,N", [(3, 70, 90), (50, 70, 90), (700, 300, 520), (3000, 512, 512)])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (4, 4), (6, 2), (3, 3), (1000, 0)])
def test_wgrad_strides_and_alignment(fmt, T, D, N, pad, offset, algo):
    q, x, dy = wgrad_case(np.random.default_rng(pad + offset), T, D, N, fmt)
    view, _ = matrix(dy, pad, offset)
    out, buf = matrix(np.zeros((D, N)), pad, offset)
    assert g.q8_wgrad(q, view, out=out, algo=algo) is out
    assert_wgrad(out, x, dy)
    assert outside_is_nan(out, buf)


@pytest.mark.parametrize("T,D,N", [(20, 40, 50), (500, 260, 300), (8192, 128, 260),
                                   (4100, 1281, 2049)])
@pytest.mark.parametrize("alpha,beta", [(1.0, 1.0), (0.5, 0.0), (-2.0, 0.25), (1.0, -1.0)])
def test_wgrad_alpha_beta(T, D, N, alpha, beta):
    rng = np.random.default_rng(T)
    q, x, dy = wgrad_case(rng, T, D, N, "int8")
    old = rng.standard_normal((D, N)).astype(np.float32)
    out, buf = matrix(old, 3)
    g.q8_wgrad(q, matrix(dy)[0], out=out, alpha=alpha, beta=beta)
    assert_wgrad(out, x, dy, alpha, beta, old)
    assert outside_is_nan(out, buf)


@pytest.mark.parametrize("T,D,N", [(20, 40, 50), (500, 260, 300), (8192, 128, 260)])
def test_wgrad_without_beta_ignores_what_was_there(T, D, N):
    q, x, dy = wgrad_case(np.random.default_rng(T), T, D, N, "e4m3")
    out, _ = matrix(np.full((D, N), np.nan))
    g.q8_wgrad(q, matrix(dy)[0], out=out)
    assert_wgrad(out, x, dy)


def test_wgrad_of_no_tokens_and_of_alpha_zero():
    torch = t()
    old = torch.randn(40, 30, device="cuda")
    empty = g.q8_empty(0, 40)
    dy0 = torch.empty(0, 30, device="cuda")
    assert bool((g.q8_wgrad(empty, dy0) == 0).all())
    out = old.clone()
    g.q8_wgrad(empty, dy0, out=out, beta=0.5)
    assert bool((out == 0.5 * old).all())
    q, _ = checkpoint(np.full((9, 40), np.nan, dtype=np.float32), "int8")
    nan = torch.full((9, 30), float("nan"), device="cuda")
    g.q8_wgrad(q, nan, out=out, alpha=0.0, beta=2.0)
    assert bool((out == old).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,D,N", [(40, 70, 90), (700, 300, 520), (9000, 100, 64)])
def test_wgrad_keeps_non_finite_values_to_their_rows_and_columns(fmt, T, D, N):
    rng = np.random.default_rng(T)
    x = _q8.activations(rng, T, D)
    x[T // 2, 40] = np.inf
    q, xv = checkpoint(x, fmt)
    dy = rng.standard_normal((T, N)).astype(np.float32)
    dy[T - 1, N - 1] = np.nan
    dy[0, 3] = np.inf
    got = g.q8_wgrad(q, matrix(dy)[0]).cpu().numpy()
    bad = np.zeros((D, N), dtype=bool)
    bad[32:64] = True
    bad[:, [3, N - 1]] = True
    assert np.array_equal(~np.isfinite(got), bad)


@pytest.mark.parametrize("T,D,N", [(64, 96, 64), (600, 300, 520), (20000, 256, 256)])
def test_wgrad_runs_alike_every_time(T, D, N):
    q, _, dy = wgrad_case(np.random.default_rng(T), T, D, N, "int8")
    dev, _ = matrix(dy)
    first = g.q8_wgrad(q, dev)
    for _ in range(5):
        assert bool((g.q8_wgrad(q, dev) == first).all())


def test_wgrad_against_differences_of_the_product():
    """The loss sum(dY * (X^ W)) is linear in W: its difference along a direction E is <dW, E>."""
    torch = t()
    rng = np.random.default_rng(8)
    q, x, dy = wgrad_case(rng, 300, 100, 60, "int8")
    dy_dev, _ = matrix(dy)
    dw = g.q8_wgrad(q, dy_dev).double()
    xv = g.q8_restore(q)
    for _ in range(4):
        w = torch.from_numpy(rng.standard_normal((100, 60)).astype(np.float32)).cuda()
        e = torch.from_numpy(rng.standard_normal((100, 60)).astype(np.float32)).cuda()

        def loss(m):
            return (dy_dev.double() * g.matmul(xv, m).double()).sum()

        diff = (loss(w + e) - loss(w - e)) / 2
        size = float((dy_dev.double().abs() * (xv.double().abs() @ e.double().abs())).sum())
        # fp32 products of 100 terms and the shifted weights' roundings
        assert abs(float(diff - (dw * e.double()).sum())) <= 1e-5 * size


# ---- streams, graphs, offsets, refusals -------------------------------------------------------------


def test_calls_on_another_stream():
    torch = t()
    rng = np.random.default_rng(2)
    x = _q8.activations(rng, 600, 512)
    dy = rng.standard_normal((600, 320)).astype(np.float32)
    dev_x, dev_dy = matrix(x)[0], matrix(dy)[0]
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        q = g.q8_store(dev_x, stream=side)
        back = g.q8_restore(q, stream=side)
        dw = g.q8_wgrad(q, dev_dy, stream=side)
        h, gq, uq = g.q8_gated(dev_x, dev_x, stream=side)
        dg, du, hq = g.q8_gated_backward(gq, uq, dev_x, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        codes, exps = _q8.store(x, "int8")
        want = _q8.values(codes, exps, "int8")
        assert np.array_equal(back.double().cpu().numpy(), want)
        assert_wgrad(dw, want, dy)
        assert torch.equal(g.q8_gated(dev_x, dev_x)[0], h)
        assert torch.equal(g.q8_gated_backward(gq, uq, dev_x)[0], dg)


@pytest.mark.parametrize("T,D,N", [(48, 64, 96), (600, 512, 320), (16384, 256, 256), (700, 300, 301)])
def test_captured_step_replays_on_new_inputs(T, D, N):
    torch = t()
    rng = np.random.default_rng(4)
    x = torch.from_numpy(_q8.activations(rng, T, D)).cuda()
    dy = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).cuda()
    q = g.q8_empty(T, D)
    dw = torch.empty(D, N, device="cuda")

    def step():
        g.q8_store(x, out=q)
        g.q8_wgrad(q, dy, out=dw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        x.copy_(torch.from_numpy(_q8.activations(rng, T, D)))
        dy.copy_(torch.randn(T, N, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = dw.clone()
        step()
        assert torch.equal(got, dw)


def test_offsets_beyond_32_bits():
    """Rows more than 2^31 elements apart, in every operand that may have such a stride."""
    torch = t()
    far = 2 ** 30 + 4
    rows, cols, N = 3, 65, 40
    rng = np.random.default_rng(6)
    x, dy = _q8.activations(rng, rows, cols), rng.standard_normal((rows, N)).astype(np.float32)
    buf = torch.empty(2 * far + 256, device="cuda")
    wide = buf.as_strided((rows, cols), (far, 1))
    wide.copy_(torch.from_numpy(x))
    raw = torch.empty(2 * (2 ** 31 + 16) + 256, dtype=torch.uint8, device="cuda")
    codes = raw.as_strided((rows, 80), (2 ** 31 + 16, 1))
    scales = raw.as_strided((rows, 16), (2 ** 31 + 16, 1), 128)
    q = g.Q8(codes, scales, cols)
    g.q8_store(wide, out=q)
    want_codes, want_exps = _q8.store(x, "int8")
    got_codes, got_exps = bytes_of(q)
    assert np.array_equal(got_codes, want_codes) and np.array_equal(got_exps, want_exps)
    v = _q8.values(want_codes, want_exps, "int8")
    out = buf.as_strided((rows, cols), (far, 1), 128)
    g.q8_restore(q, out=out)
    assert np.array_equal(out.double().cpu().numpy(), v)
    dyw = buf.as_strided((rows, N), (far, 1))
    dyw.copy_(torch.from_numpy(dy))
    assert_wgrad(g.q8_wgrad(q, dyw), v, dy)
    h, gq, uq = g.q8_gated(wide, out)
    w2, o2 = wide.clone(), out.clone()
    assert torch.equal(h, g.q8_gated(w2, o2)[0])


def test_many_elements():
    """More than 2^31 elements and codes in one matrix."""
    torch = t()
    rows, cols = 2 ** 17 + 3, 2 ** 14 + 32
    x = torch.zeros(rows, cols, device="cuda")
    x[-2:] = torch.arange(cols, device="cuda") % 255 - 127
    q = g.q8_store(x)
    del x
    back = g.q8_restore(q, dtype=torch.bfloat16)
    want = (torch.arange(cols, device="cuda") % 255 - 127).bfloat16()
    assert bool((back[:-2] == 0).all()) and bool((back[-2:] == want).all())


def test_wgrad_with_more_than_2_31_outputs():
    torch = t()
    T, D, N = 8, 66000, 33000
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-100, 101, (T, D), generator=gen, device="cuda").float()
    dy = torch.randint(-50, 51, (T, N), generator=gen, device="cuda").float()
    q = g.q8_store(x)
    xv = g.q8_restore(q).double()
    dw = g.q8_wgrad(q, dy)
    for rows in (slice(0, 300), slice(32700, 32900), slice(65000, 66000)):  # 2^31 / N = 65075
        assert torch.equal(dw[rows].double(), xv[:, rows].t() @ dy.double())


def test_wgrad_with_more_than_2_31_codes():
    torch = t()
    T, D, N = 140000, 16416, 24
    q = g.q8_store(torch.zeros(T, D, device="cuda"))
    x = torch.arange(D, device="cuda") % 255 - 127.0
    tail = g.q8_store(x.expand(3, D).contiguous())
    q.codes[-3:] = tail.codes
    q.scales[-3:] = tail.scales
    dy = torch.ones(T, N, device="cuda")
    want = 3 * g.q8_restore(tail)[0]
    assert torch.equal(g.q8_wgrad(q, dy), want[:, None].expand(D, N))


def test_binding_refuses():
    torch = t()
    x = torch.zeros(8, 64, device="cuda")
    q = g.q8_store(x)
    for call in (
            lambda: g.q8_store(x, format="e5m2"),
            lambda: g.q8_store(x.t()),
            lambda: g.q8_store(x.half()),
            lambda: g.q8_store(x[0]),
            lambda: g.q8_store(x, out=g.q8_empty(8, 63)),
            lambda: g.q8_store(x, format="e4m3", out=q),
            lambda: g.q8_store(x[:1].expand(8, 64)),
            lambda: g.q8_restore(q, out=torch.zeros(8, 65, device="cuda")),
            lambda: g.q8_restore(q, dtype=torch.float16),
            lambda: g.q8_wgrad(q, torch.zeros(7, 5, device="cuda")),
            lambda: g.q8_wgrad(q, torch.zeros(8, 5, device="cuda"), beta=1.0),
            lambda: g.q8_wgrad(q, torch.zeros(8, 5, device="cuda"),
                               out=torch.zeros(5, 64, device="cuda")),
            lambda: g.q8_gated(x, x[:, :63]),
            lambda: g.q8_gated(x, x, act="relu"),
            lambda: g.q8_gated_backward(q, g.q8_store(x, format="e4m3"), x),
            lambda: g.q8_gated_backward(q, q, x, want_h=False, h_q=g.q8_empty(8, 64)),
            lambda: g.Q8(q.codes, q.scales, 65),
            lambda: g.Q8(q.codes[:, 1:], q.scales, 60),
            lambda: g.Q8(torch.zeros(8, 60, dtype=torch.uint8, device="cuda"), q.scales, 60)):
        with pytest.raises(ValueError):
            call()
    # what only the library can see
    with pytest.raises(g.GemmError):
        g.q8_gated(x, x.clone(), out=x)
    with pytest.raises(g.GemmError):
        g.q8_gated_backward(q, g.q8_store(x), x, h_q=q)


def test_checkpoints_made_together_are_apart():
    """The two checkpoints of a gated unit share one allocation: their bytes must not."""
    torch = t()
    gate, up = torch.randn(5, 70, device="cuda"), torch.randn(5, 70, device="cuda")
    _, gq, uq = g.q8_gated(gate, up)
    assert gq.codes.shape == uq.codes.shape == (5, 80) and gq.scales.shape == (5, 16)
    for q, x in ((gq, gate), (uq, up)):
        assert torch.equal(g.q8_restore(q), g.q8_restore(g.q8_store(x)))
        again = g.Q8(q.codes, q.scales, 70)
        assert torch.equal(g.q8_restore(again), g.q8_restore(q))


@pytest.mark.parametrize("kind,status", [(g.INJECT_WORKSPACE, g.ERR_WORKSPACE),
                                         (g.INJECT_DESCRIPTOR, g.ERR_DESCRIPTOR)])
def test_wgrad_reports_a_host_failure_and_recovers(kind, status):
    """A workspace that cannot be had, a descriptor that is refused: the status, dW as it was."""
    torch = t()
    q, x, dy = wgrad_case(np.random.default_rng(1), 4096, 300, 300, "int8")  # shares its tiles
    dev, _ = matrix(dy)
    out = torch.full((300, 300), 7.0, device="cuda")
    g.check(g.gemm_f32_release())
    g.gemm_f32_inject_host_fault(kind)
    with pytest.raises(g.GemmError) as e:
        g.q8_wgrad(q, dev, out=out)
    assert e.value.status == status
    assert bool((out == 7.0).all())
    assert_wgrad(g.q8_wgrad(q, dev, out=out), x, dy)


def test_wgrad_needs_its_workspace_before_a_capture():
    torch = t()
    q, x, dy = wgrad_case(np.random.default_rng(1), 4096, 300, 300, "int8")
    dev, _ = matrix(dy)
    out = torch.empty(300, 300, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g.check(g.gemm_f32_release())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st = g.gemm_f32_q8_wgrad(q.struct, dev.data_ptr(), 300, 300, 1.0, 0.0, out.data_ptr(), 300,
                                 stream=torch.cuda.current_stream().cuda_stream)
        out.zero_()  # a graph of something
    assert st == g.ERR_CAPTURE
    assert_wgrad(g.q8_wgrad(q, dev), x, dy)


def test_checkpoint_memory_lives_as_long_as_it_is_used():
    """Views keep the memory; dropped checkpoints give it back; empty ones have none."""
    torch = t()
    x = torch.randn(1000, 4096, device="cuda")
    q = g.q8_store(x)
    want = g.q8_restore(q).clone()
    codes, scales = q.codes, q.scales
    del q
    junk = [g.q8_store(torch.zeros(1000, 4096, device="cuda")) for _ in range(4)]
    assert torch.equal(g.q8_restore(g.Q8(codes, scales, 4096)), want)
    del junk, codes, scales
    torch.cuda.synchronize()
    gc.collect()
    before = torch.cuda.memory_allocated()
    for _ in range(50):
        g.q8_store(x)
    assert torch.cuda.memory_allocated() == before
    none = g.q8_empty(0, 70)
    assert none.codes.shape == (0, 80) and none.scales.shape == (0, 16) and none.nbytes == 0


def test_checkpoint_dropped_while_another_stream_reads_it():
    """Its memory is not handed out again before that stream is done."""
    torch = t()
    x = torch.randn(4096, 4096, device="cuda")
    want = g.q8_restore(g.q8_store(x)).clone()
    side = torch.cuda.Stream()
    for _ in range(10):
        q = g.q8_store(x)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000000)  # the reader is late
        back = g.q8_restore(q, stream=side)
        del q
        others = [g.q8_store(torch.zeros_like(x)) for _ in range(3)]
        side.synchronize()
        assert torch.equal(back, want)
        del others


def step(torch, x, gate, up, dh, dy):
    """Every operator once as a user calls it, and what each gives."""
    q = g.q8_store(x, format="e4m3")
    h, gq, uq = g.q8_gated(gate, up, act="gelu")
    dgate, dup, hq = g.q8_gated_backward(gq, uq, dh, act="gelu")
    nothing = g.q8_gated_backward(gq, uq, dh, act="gelu", want_h=False)[2]
    assert nothing is None and q.format == "e4m3" and hq.format == gq.format == "int8"
    assert (q.rows, q.cols, q.device) == (x.shape[0], x.shape[1], x.get_device())
    assert repr(q) == f"Q8({x.shape[0]} x {x.shape[1]}, e4m3)"
    again = g.Q8(q.codes, q.scales, q.cols, format="e4m3")
    return [h, dgate, dup, g.q8_restore(again), g.q8_restore(hq, dtype=torch.bfloat16),
            g.q8_wgrad(again, dy), g.q8_restore(gq), g.q8_restore(uq)]


@pytest.mark.parametrize("rows,cols", [(0, 33), (1, 33), (5, 0), (1, 1), (64, 512), (37, 1001)])
def test_calls_with_and_without_the_native_module(monkeypatch, rows, cols):
    """The binding's two ways through a call give the same bits."""
    torch = t()
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    wide = torch.randn(rows, 2 * cols + 3, device="cuda", generator=gen)
    x, gate, up = wide[:, :cols], wide[:, :cols], wide[:, cols:2 * cols]
    dh = torch.randn(rows, cols, device="cuda", generator=gen)
    dy = torch.randn(rows, 40, device="cuda", generator=gen)
    want = step(torch, x, gate, up, dh, dy)
    assert _binding._native is not None
    monkeypatch.setattr(_binding, "_native", None)
    got = step(torch, x, gate, up, dh, dy)
    for a, b in zip(want, got):
        assert a.shape == b.shape and a.dtype == b.dtype and a.stride() == b.stride()
        assert torch.equal(a, b)


def test_native_module_takes_only_plain_tensors():
    """A parameter, a double, a transpose, host memory: each by the other way, with its answer."""
    torch = t()
    x = torch.randn(70, 70, device="cuda")
    want = g.q8_restore(g.q8_store(x))
    assert torch.equal(g.q8_restore(g.q8_store(torch.nn.Parameter(x))), want)
    for bad in (x.double(), x.t(), x.cpu(), x[0], x[:1].expand(8, 70)):
        for call in (lambda: g.q8_store(bad), lambda: g.q8_gated(bad, bad),
                     lambda: g.q8_wgrad(g.q8_store(x), bad)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        g.q8_store(x, format="int4")
    q = g.q8_store(x)
    with pytest.raises(ValueError):
        g.q8_gated_backward(q, q, x, act="relu")


def test_native_module_reports_the_librarys_status():
    torch = t()
    q, x, dy = wgrad_case(np.random.default_rng(1), 4096, 300, 300, "int8")
    dev, _ = matrix(dy)
    g.check(g.gemm_f32_release())
    g.gemm_f32_inject_host_fault(g.INJECT_WORKSPACE)
    with pytest.raises(g.GemmError) as e:
        g.q8_wgrad(q, dev)
    assert e.value.status == g.ERR_WORKSPACE
    assert_wgrad(g.q8_wgrad(q, dev), x, dy)
