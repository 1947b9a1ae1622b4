"""cudaStreamPerThread: one handle for a stream of every host thread, whose calls run beside one another."""

import threading

import pytest

import dense_fp32_gemm_row_gb300 as g
from tests.test_graph_workspace_gpu import HostProduct, SplitProduct, WeightGradient
from tests import _gpu

pytestmark = pytest.mark.gpu


class PerThread:
    """The stream as the cases take one."""

    cuda_stream = 2  # the value of cudaStreamPerThread


@pytest.fixture(autouse=True)
def _release():
    yield
    _gpu.torch().cuda.synchronize()
    g.check(g.gemm_f32_device_status(1), "device status")
    g.gemm_f32_release()


def in_threads(work, cases):
    """work(case) for each case in a thread of its own, all at once."""
    t = _gpu.torch()
    errors, gate = [], threading.Barrier(len(cases))

    def run(case):
        try:
            t.cuda.set_device(0)
            gate.wait(60)
            work(case)
        except Exception as e:  # reported by the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=(case,)) for case in cases]
    for x in threads:
        x.start()
    for x in threads:
        x.join(120)
    t.cuda.synchronize()
    assert not errors and not any(x.is_alive() for x in threads), errors


def small_host_product(seed):
    return HostProduct(seed, (2304, 1100, 1024))


@pytest.mark.parametrize("kind", [WeightGradient, SplitProduct, small_host_product])
def test_threads_share_no_buffers(kind):
    t = _gpu.torch()
    cases = [kind(seed) for seed in range(4)]
    want = []
    for case in cases:
        case.call(t.cuda.current_stream())
        t.cuda.synchronize()
        want.append(case.out.clone())
        case.out.fill_(float("nan"))
    t.cuda.synchronize()

    def work(case):
        for _ in range(20):
            case.call(PerThread)

    for _ in range(5):
        in_threads(work, cases)
        for case, w in zip(cases, want):
            assert t.equal(case.out, w)
            case.out.fill_(float("nan"))
        t.cuda.synchronize()


def test_what_ended_threads_held_is_given_back():
    t = _gpu.torch()
    cases = [WeightGradient(1)]
    t.cuda.synchronize()
    t.cuda.empty_cache()
    start = t.cuda.mem_get_info()[0]
    for _ in range(12):
        in_threads(lambda case: case.call(PerThread), cases)
    # the last thread's, and room for what CUDA keeps of a thread
    assert start - t.cuda.mem_get_info()[0] < 3 * WeightGradient.bytes
