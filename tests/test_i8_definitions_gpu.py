"""The 8-bit integer layers against what they stand for: values of codes and scales, and activations
far from zero."""

import numpy as np
import pytest

import dense_fp32_gemm_row_gb300 as g
from tests import _i8, _q8
from tests.test_i8_gpu import activations, down, dtype, quiet, t, up

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -23


def gates() -> np.ndarray:
    """Both signs, all sizes; close together around where e^88 ends fp32 and where gelu's exponential
    does."""
    a = np.concatenate([np.geomspace(1e-30, 1.0, 40), np.linspace(1.0, 12.0, 90), np.linspace(12.0, 15.0, 31),
                        np.linspace(15.0, 86.0, 72), np.linspace(86.0, 90.0, 161), np.linspace(90.0, 111.0, 22),
                        [1e3, 1e10, 1e30]]).astype(np.float32).astype(np.float64)
    return np.concatenate([[0.0], a, -a])


@pytest.mark.parametrize("T", [1, 3, 20, 40, 200])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_far_from_zero(T, act):
    """Gates that are exact, so that nothing but the activation's own error is allowed: that of its
    steps, in multiples of its value, and what fp32 does not hold.  Up is 3, a product's rounding."""
    torch = t()
    z = gates()
    one = g.i8_empty(T, 1)
    one.codes.fill_(1)
    one.scales.fill_(1.0)
    w, v = g.i8_empty(len(z), 1), g.i8_empty(len(z), 1)
    for m, s in ((w, z), (v, np.full(len(z), 3.0))):
        m.codes.fill_(1)
        m.scales.copy_(torch.from_numpy(s.astype(np.float32)))
    got = down(g.i8_gated(one, w, v, act=act)).astype(np.float64)
    quiet()
    a = _q8.act(z, act)[0]
    # silu: expf 2 ulp, the sum half an ulp, the quotient 2, 4.5 in all.  gelu: the function's 4 and
    # the exponential's 2 and the rounded z^2 / 2, which the exponential makes z^2 / 2 halves of an ulp of
    # its value; products and the rest of it 2.
    steps = 5.0 if act == "silu" else 8.0 + z * z / 2
    # silu of gates from -87.33 to -104: 0 for up to 1.03e-36; gelu's below the normal numbers: z times one
    lost = np.where((z < -87.3) & (z > -111), 1.03e-36, 0.0) if act == "silu" else \
        np.where((z < -12.0) & (z > -15.0), np.abs(z) * 2.0 ** -126, 0.0)
    want = 3.0 * a
    bound = 3.0 * (steps * ULP * np.abs(a) + lost) * (1 + ULP) + ULP / 2 * np.abs(want) + 2.0 ** -149
    assert np.all(np.abs(got - want) <= bound)
    gone = z <= (-111 if act == "silu" else -15)
    assert gone.any() and np.all(got[:, gone] == 0.0)


@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (9, 257), (1, 4096), (700, 130), (310, 1024), (40, 5001),
                                       (4, 16384), (2, 20000)])
def test_values_of_stored_rows(rows, cols, name):
    """Within half a step: what code = z (127 / a) loses before it is rounded are two roundings, and
    a / 127 one, each half an ulp of the value."""
    rng = np.random.default_rng(rows + 13 * cols)
    x = activations(rng, rows, cols, name)
    q = g.i8_store(up(x, name))
    quiet()
    scale = down(q.scales).astype(np.float64)[:, None]
    value = down(q.codes)[:, :cols] * scale
    assert np.all(np.abs(value - x) <= 0.5 * scale + 3.01 * ULP / 2 * np.abs(x))


@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (9, 257), (1, 4096), (700, 130), (310, 1024), (40, 5001),
                                       (4, 16384), (2, 20000)])
def test_values_of_the_norm(rows, cols, residual, name):
    """code * scale against s w / sqrt(mean s^2 + eps): half a step, the two roundings of z (127 / a),
    and the scale's own error, which counts z's."""
    torch = t()
    rng = np.random.default_rng(rows + 17 * cols)
    x = activations(rng, rows, cols, name)
    r = activations(rng, rows, cols, name) if residual else None
    w = down(torch.from_numpy(rng.standard_normal(cols).astype(np.float32)).to(dtype(name)))
    w[cols // 2:cols // 2 + 1] = 0.0 if cols > 1 else 0.5
    eps = float(np.float32(1e-3))
    q, _ = g.i8_norm(up(x, name), up(w[None], name)[0], residual=up(r, name) if residual else None, eps=eps)
    quiet()
    s = x.astype(np.float64) + (r if residual else 0.0)
    want = s * w / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    scale = down(q.scales).astype(np.float64)[:, None]
    value = down(q.codes)[:, :cols] * scale
    assert np.all(np.abs(value - want) <= 0.5 * scale + (_i8.norm_bound(cols) + 4 * ULP / 2) * np.abs(want))
