"""The 8-bit integer layers against what they stand for: values of codes and scales, and activations
far from zero."""

import numpy as np
import pytest

import dense_fp32_gemm_row_gb300 as g
from tests import _q8
from tests.test_i8_gpu import down, quiet, t

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
