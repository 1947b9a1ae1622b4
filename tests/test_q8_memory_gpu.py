"""A checkpoint whose tensors are given other memory: activations moved to the host and back, freed
between the passes, or exchanged."""

import pytest

import dense_fp32_gemm_row_gb300 as g
from dense_fp32_gemm_row_gb300 import q8 as binding

pytestmark = pytest.mark.gpu

SHAPES = [(1, 70), (300, 200)]  # the native module leaves single rows to the other way


def t():
    import torch
    return torch


@pytest.fixture(params=["native", "python"])
def way(request, monkeypatch):
    binding._load_torch()
    assert binding._native is not None
    if request.param == "python":
        monkeypatch.setattr(binding, "_native", None)


def made(rows, cols):
    """Checkpoints as the operators make them, and of a user's tensors; the values of each."""
    torch = t()
    x = torch.randn(rows, cols, device="cuda")
    q = g.q8_store(x)
    codes, scales = q.codes.clone(), q.scales.clone()
    return [q, g.Q8(codes, scales, cols)], g.q8_restore(q)


def calls(q, x):
    return (lambda: g.q8_restore(q), lambda: g.q8_wgrad(q, x), lambda: g.q8_store(x, out=q),
            lambda: g.q8_gated_backward(q, q, x), lambda: q.struct)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_freed_memory_is_not_read(way, rows, cols):
    torch = t()
    for q in made(rows, cols)[0]:
        held = [s.clone() for s in (q.codes, q.scales)]
        storages = [s.untyped_storage() for s in (q.codes, q.scales)]
        size = [s.nbytes() for s in storages]
        for s in storages:
            s.resize_(0)
        x = torch.ones(rows, cols, device="cuda")
        for call in calls(q, x):
            with pytest.raises(ValueError):
                call()
        for s, n in zip(storages, size):
            s.resize_(n)
        q.codes.copy_(held[0])
        q.scales.copy_(held[1])
        assert torch.equal(g.q8_restore(q), g.q8_restore(g.Q8(*held, cols)))


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_memory_that_moved_is_followed(way, rows, cols):
    torch = t()
    qs, want = made(rows, cols)
    x = torch.randn(rows, cols, device="cuda")
    dw = g.q8_wgrad(qs[0], x)
    for q in qs:
        for s in (q.codes, q.scales):
            s.untyped_storage().resize_(s.untyped_storage().nbytes() + (8 << 20))
        junk = [torch.full((64,), 1e9, device="cuda") for _ in range(2000)]
        assert torch.equal(g.q8_restore(q), want) and torch.equal(g.q8_wgrad(q, x), dw)
        del junk


def test_tensors_exchanged(way):
    torch = t()
    (_, q), want = made(300, 200)
    other = g.q8_store(torch.randn(300, 200, device="cuda"))
    assert not torch.equal(g.q8_restore(other), want)
    q.codes.data, q.scales.data = other.codes, other.scales
    assert torch.equal(g.q8_restore(q), g.q8_restore(other))
    q.codes.data = other.codes[:200]
    with pytest.raises(ValueError):
        g.q8_restore(q)
