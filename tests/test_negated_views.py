"""Views whose memory holds their values with the other sign, as torch makes them of the imaginary
part of a conjugate: refused, where their memory would have been taken for the values."""

import pytest

import dense_fp32_gemm_row_gb300 as g
from tests.test_i8_abi import Vector, lib, loaded, weight  # noqa: F401
from tests.test_q8_binding import Memory

torch = pytest.importorskip("torch")


class Negated(Memory):
    def is_neg(self):
        return True

    def is_contiguous(self):
        return True


class NegatedVector(Vector, Negated):
    pass


class Plain(Memory):
    def is_contiguous(self):
        return True


def test_stand_ins_without_a_gpu():
    shape = (8, 64)
    x, neg = Plain(shape, torch.float32), Negated(shape, torch.float32)
    codes, scales = Memory(shape, torch.int8), Vector((8,), torch.float32)
    bytes, exponents = Memory(shape, torch.uint8), Memory((8, 16), torch.uint8)
    q, c = g.I8(codes, scales, 64), g.Q8(bytes, exponents, 64)
    square = Plain((64, 64), torch.float32)
    for call in (lambda: g.i8_store(neg), lambda: g.i8_norm(neg, weight(64)),
                 lambda: g.i8_norm(x, NegatedVector((64,), torch.float32)),
                 lambda: g.i8_norm(x, weight(64), residual=neg),
                 lambda: g.I8(Negated(shape, torch.int8), scales, 64),
                 lambda: g.I8(codes, NegatedVector((8,), torch.float32), 64),
                 lambda: g.i8_matmul(q, q, out=Negated((8, 8), torch.float32)),
                 lambda: g.q8_store(neg), lambda: g.q8_wgrad(c, neg), lambda: g.q8_gated(x, neg),
                 lambda: g.q8_restore(c, out=neg), lambda: g.q8_gated_backward(c, c, neg),
                 lambda: g.Q8(Negated(shape, torch.uint8), exponents, 64),
                 lambda: g.Q8(bytes, Negated((8, 16), torch.uint8), 64),
                 lambda: g.matmul(neg, square), lambda: g.matmul(x, Negated((64, 64), torch.float32)),
                 lambda: g.matmul(x, square, out=neg)):
        with pytest.raises(ValueError, match="negated"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("module", [True, False])
def test_tensors(module, monkeypatch):
    import dense_fp32_gemm_row_gb300.i8 as i8
    import dense_fp32_gemm_row_gb300.q8 as q8

    g.i8_store(torch.ones(1, 1, device="cuda"))
    assert i8._native is not None and q8._native is not None
    if not module:
        monkeypatch.setattr(i8, "_native", None)
        monkeypatch.setattr(q8, "_native", None)
    column = torch.complex(torch.ones(5, 1), torch.arange(1.0, 6.0)[:, None]).cuda().conj().imag
    one = torch.complex(torch.ones(1, 1), torch.ones(1, 1)).cuda().conj().imag
    wide = torch._neg_view(torch.randn(5, 40, device="cuda"))
    x, w = torch.randn(5, 40, device="cuda"), torch.ones(40, device="cuda")
    q, c = g.i8_store(x), g.q8_store(x)
    assert column.is_neg() and one.is_neg() and wide.is_neg() and one.is_contiguous()
    for call in (lambda: g.i8_store(column), lambda: g.i8_store(wide), lambda: g.i8_norm(wide, w),
                 lambda: g.i8_norm(x, torch._neg_view(w)), lambda: g.i8_norm(x, w, residual=wide),
                 lambda: g.i8_norm(x, w, residual=x, total=wide),
                 lambda: g.I8(torch._neg_view(q.codes), q.scales, 40),
                 lambda: g.I8(q.codes, torch._neg_view(q.scales), 40),
                 lambda: g.i8_matmul(q, q, out=torch._neg_view(torch.empty(5, 5, device="cuda"))),
                 lambda: g.q8_store(column), lambda: g.q8_store(wide), lambda: g.q8_gated(x, wide),
                 lambda: g.q8_wgrad(c, wide), lambda: g.q8_gated_backward(c, c, wide),
                 lambda: g.q8_restore(c, out=wide), lambda: g.Q8(torch._neg_view(c.codes), c.scales, 40),
                 lambda: g.matmul(one, one), lambda: g.matmul(x, torch._neg_view(x.t().contiguous()))):
        with pytest.raises(ValueError, match="negated"):
            call()
    # what the refusal says to do
    assert torch.equal(g.i8_store(wide.resolve_neg()).codes[:, :40], g.i8_store(-wide.neg()).codes[:, :40])
    assert torch.equal(g.i8_store(column.resolve_neg()).codes[:, 0], torch.full((5,), -127, dtype=torch.int8, device="cuda"))
    # codes turned into a view after the matrix was made
    q.codes = torch._neg_view(q.codes)
    with pytest.raises(ValueError, match="negated"):
        g.i8_matmul(q, q)
