"""What the 8-bit operators' Python binding refuses before any call of the library, without a GPU."""

import pytest

import dense_fp32_gemm_row_gb300 as g
from dense_fp32_gemm_row_gb300 import build as gbuild
from dense_fp32_gemm_row_gb300 import q8

torch = pytest.importorskip("torch")

WIDE = 2 ** 32 + 8  # as an int of 32 bits: 8


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    q8._load_torch()


class Memory:
    """As much of a CUDA tensor as the binding looks at, of any size and without memory."""

    is_cuda = True

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.index = shape, dtype, device

    def dim(self):
        return 2

    def stride(self):
        return self.shape[1], 1

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x7000_0000_0000

    def numel(self):
        return self.shape[0] * self.shape[1]

    def storage_offset(self):
        return 0

    def untyped_storage(self):
        return self

    def nbytes(self):
        return self.numel() * self.dtype.itemsize


def floats(rows, cols):
    return Memory((rows, cols), torch.float32)


def checkpoint(rows, cols):
    return g.Q8(Memory((rows, -(-cols // 16) * 16), torch.uint8),
                Memory((rows, -(-cols // 512) * 16), torch.uint8), cols)


def test_a_stream_of_another_device():
    """Entering it would make its device the current one, and the call run on the other's stream."""
    class Stream:
        device = torch.device("cuda", 1)

    x, q = floats(8, 64), checkpoint(8, 64)
    for call in (lambda: g.q8_store(x, stream=Stream), lambda: g.q8_restore(q, stream=Stream),
                 lambda: g.q8_wgrad(q, x, stream=Stream), lambda: g.q8_gated(x, x, stream=Stream),
                 lambda: g.q8_gated_backward(q, q, x, stream=Stream)):
        with pytest.raises(ValueError, match="stream"):
            call()


# ---- sizes that the library's 32-bit arguments cannot hold ----------------------------------------


@pytest.mark.parametrize("size", [2 ** 31, WIDE])
def test_matrices_beyond_32_bits(size):
    q = checkpoint(1, 1)
    for call in (lambda: g.q8_store(floats(size, 1)), lambda: g.q8_store(floats(1, size)),
                 lambda: g.q8_wgrad(q, floats(1, size)),
                 lambda: g.q8_gated(floats(1, size), floats(1, size)),
                 lambda: g.q8_gated_backward(q, q, floats(size, 1)),
                 lambda: g.q8_restore(q, out=floats(size, 1))):
        with pytest.raises(ValueError, match=r"2\^31"):
            call()


@pytest.mark.parametrize("size", [2 ** 31, WIDE])
def test_checkpoints_beyond_32_bits(size):
    for call in (lambda: checkpoint(size, 1), lambda: checkpoint(1, size),
                 lambda: g.q8_empty(size, 1), lambda: g.q8_empty(1, size)):
        with pytest.raises(ValueError, match=r"2\^31"):
            call()
    assert checkpoint(2 ** 31 - 1, 1).struct.rows == 2 ** 31 - 1


def test_product_beyond_32_bits():
    class Contiguous(Memory):
        def is_contiguous(self):
            return True

    def f(rows, cols):
        return Contiguous((rows, cols), torch.float32)

    for a, b in ((f(WIDE, 1), f(1, 1)), (f(1, 1), f(1, WIDE)), (f(1, WIDE), f(WIDE, 1))):
        with pytest.raises(ValueError, match=r"2\^31"):
            g.matmul(a, b)
    with pytest.raises(ValueError, match=r"2\^31"):
        g.matmul(f(1, 1), f(1, 1), splits=2 ** 32 + 1)


def test_raw_arguments_beyond_32_bits():
    q = g.Q8Struct(0x7000_0000_0000, 0x7100_0000_0000, 16, 16, 1, 1, 0)
    for N, splits in ((WIDE, 0), (-WIDE, 0), (8, 2 ** 32 + 1)):
        assert g.gemm_f32_q8_wgrad(q, 0x7200_0000_0000, WIDE, N, 1.0, 0.0, 0x7300_0000_0000, WIDE, 0,
                                   splits) == g.ERR_INVALID_VALUE
    with pytest.raises(ValueError, match=r"2\^31"):
        g.q8_wgrad(checkpoint(1, 1), floats(1, 1), algo="3xbf16", splits=2 ** 32 + 1)
    for rows, cols in ((WIDE, 1), (1, WIDE)):
        with pytest.raises(ValueError, match=r"2\^31"):
            g.Q8Struct(0, 0, 16, 16, rows, cols, 0)
