"""Graphs replayed beside one another and beside calls on the stream of their capture.

Partial sums and padded copies lie in device memory of the library's.  Nothing orders the replays of
two graphs, or a replay and a call on the stream that the graph was captured from, so each graph needs
memory of its own; and gives it back when it is destroyed, or every capture would cost that much.
"""

import gc

import pytest

import dense_fp32_gemm_row_gb300 as g
from tests import _gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _release():
    yield
    _gpu.torch().cuda.synchronize()
    g.check(g.gemm_f32_device_status(1), "device status")
    g.gemm_f32_release()


class WeightGradient:
    """dW of a 65536-token batch: 152 partial sums of 128 KB, added by a second kernel."""

    bytes = 152 * 128 * 1024

    def __init__(self, seed):
        t = _gpu.torch()
        gen = t.Generator(device="cuda").manual_seed(seed)
        self.q = g.q8_store(t.randn((65536, 256), generator=gen, device="cuda"))
        self.dy = t.randn((65536, 256), generator=gen, device="cuda")
        self.out = t.empty((256, 256), device="cuda")

    def call(self, stream):
        g.check(g.gemm_f32_q8_wgrad(self.q.struct, self.dy.data_ptr(), 256, 256, 1.0, 0.0,
                                    self.out.data_ptr(), 256, stream=stream.cuda_stream), "q8_wgrad")


class SplitProduct:
    """C = A B with eight K ranges in the workspace, added by a second kernel."""

    bytes = 8 * 256 * 256 * 4

    def __init__(self, seed, algo=g.ALGO_FFMA):
        t = _gpu.torch()
        gen = t.Generator(device="cuda").manual_seed(seed)
        self.algo = algo
        self.a = t.randn((256, 32768), generator=gen, device="cuda")
        self.b = t.randn((32768, 256), generator=gen, device="cuda")
        self.out = t.empty((256, 256), device="cuda")

    def call(self, stream):
        g.check(g.gemm_f32_algo_splitk(self.a.data_ptr(), self.b.data_ptr(), self.out.data_ptr(), 256,
                                       256, 32768, self.algo, 8, stream.cuda_stream), "splitk")


class PaddedProduct(SplitProduct):
    """The same on the tensor cores from rows that are first copied to a 16-byte stride."""

    bytes = 2 * 256 * 32768 * 4

    def __init__(self, seed):
        super().__init__(seed, g.ALGO_3XTF32)
        t = _gpu.torch()
        self.a = t.cat([t.zeros(1, device="cuda"), self.a.flatten()])[1:].view(256, 32768)


class HostProduct:
    """C = A B from host buffers through copies on the device, by row panels or by panels of K."""

    def __init__(self, seed, shape):
        t = _gpu.torch()
        gen = t.Generator().manual_seed(seed)
        self.shape = M, N, K = shape
        self.a, self.b = (t.randn(s, generator=gen).pin_memory() for s in ((M, K), (K, N)))
        self.out = t.empty((M, N)).pin_memory()

    def call(self, stream):
        g.check(g.gemm_f32_host(self.a.data_ptr(), self.b.data_ptr(), self.out.data_ptr(), *self.shape,
                                stream=stream.cuda_stream), "gemm_f32_host")


def captured(case, stream):
    t = _gpu.torch()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=stream):
        case.call(stream)
    return graph


def answers(cases, stream):
    """What each case gives by itself."""
    t = _gpu.torch()
    want = []
    for case in cases:
        case.call(stream)
        t.cuda.synchronize()
        want.append(case.out.clone())
        case.out.fill_(float("nan"))
    return want


@pytest.mark.parametrize("kind", [WeightGradient, SplitProduct, PaddedProduct])
def test_two_graphs_of_one_stream_replayed_at_once(kind):
    t = _gpu.torch()
    source, left, right = t.cuda.Stream(), t.cuda.Stream(), t.cuda.Stream()
    cases = [kind(1), kind(2)]
    want = answers(cases, source)
    graphs = [captured(case, source) for case in cases]
    for _ in range(30):
        for _ in range(4):
            for graph, stream in zip(graphs, (left, right)):
                with t.cuda.stream(stream):
                    graph.replay()
        t.cuda.synchronize()
        for case, w in zip(cases, want):
            assert t.equal(case.out, w)
            case.out.fill_(float("nan"))


@pytest.mark.parametrize("kind", [WeightGradient, SplitProduct, PaddedProduct])
def test_a_graph_replayed_beside_calls_on_its_stream(kind):
    t = _gpu.torch()
    source, other = t.cuda.Stream(), t.cuda.Stream()
    cases = [kind(3), kind(4)]
    want = answers(cases, source)
    graph = captured(cases[0], source)
    for _ in range(30):
        for _ in range(4):
            with t.cuda.stream(other):
                graph.replay()
            cases[1].call(source)
        t.cuda.synchronize()
        for case, w in zip(cases, want):
            assert t.equal(case.out, w)
            case.out.fill_(float("nan"))


@pytest.mark.parametrize("shape", [(2304, 1100, 1024), (2048, 2048, 2048)])
def test_captured_host_calls_replayed_at_once(shape):
    t = _gpu.torch()
    source, left, right = t.cuda.Stream(), t.cuda.Stream(), t.cuda.Stream()
    cases = [HostProduct(seed, shape) for seed in (1, 2, 3)]
    want = answers(cases, source)
    graphs = [captured(case, source) for case in cases[:2]]
    for _ in range(10):
        for graph, stream in zip(graphs, (left, right)):
            with t.cuda.stream(stream):
                graph.replay()
        cases[2].call(source)
        t.cuda.synchronize()
        for case, w in zip(cases, want):
            assert t.equal(case.out, w)
            case.out.fill_(float("nan"))


def test_calls_of_one_capture_share_what_a_graph_gives_back():
    t = _gpu.torch()
    source = t.cuda.Stream()
    case = WeightGradient(5)
    want, = answers([case], source)

    def free():
        gc.collect()
        t.cuda.synchronize()
        t.cuda.empty_cache()
        return t.cuda.mem_get_info()[0]

    def several():
        t.cuda.synchronize()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=source):
            for _ in range(5):
                case.call(source)
        return graph

    start = free()
    first = several()
    assert case.bytes <= start - free() < 2 * case.bytes  # memory of its own, once for its five calls
    second = several()
    both = start - free()
    assert both >= 2 * case.bytes
    del first, second
    for _ in range(10):  # taken over by the graphs that follow
        graph = several()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(case.out, want)
        case.out.fill_(float("nan"))
        del graph
        assert start - free() < both + case.bytes


def test_a_larger_call_later_in_the_capture():
    """The smaller call's memory stays its graph's; the larger call gets another piece."""
    t = _gpu.torch()
    source = t.cuda.Stream()
    cases = [SplitProduct(6), WeightGradient(7), SplitProduct(8)]
    want = answers(cases, source)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=source):
        for case in cases:
            case.call(source)
    for _ in range(3):
        graph.replay()
        t.cuda.synchronize()
        for case, w in zip(cases, want):
            assert t.equal(case.out, w)
            case.out.fill_(float("nan"))


def test_a_capture_whose_workspace_cannot_be_had():
    t = _gpu.torch()
    source = t.cuda.Stream()
    case = WeightGradient(9)
    want, = answers([case], source)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=source):
        case.out.zero_()
        g.gemm_f32_inject_host_fault(g.INJECT_WORKSPACE)
        with pytest.raises(g.GemmError) as e:
            case.call(source)
        case.out.add_(1.0)  # the capture goes on
    assert e.value.status == g.ERR_WORKSPACE
    graph.replay()
    t.cuda.synchronize()
    assert bool((case.out == 1.0).all())
    again = captured(case, source)
    again.replay()
    t.cuda.synchronize()
    assert t.equal(case.out, want)


def test_a_graph_destroyed_while_it_runs():
    """Its memory goes to no other graph before its last replay is done."""
    t = _gpu.torch()
    source, left = t.cuda.Stream(), t.cuda.Stream()
    cases = [WeightGradient(10), WeightGradient(11)]
    want = answers(cases, source)

    def late(case, cycles):
        # without the waits and the collection of torch.cuda.graph
        graph = t.cuda.CUDAGraph()
        with t.cuda.stream(source):
            graph.capture_begin()
            if cycles:
                t.cuda._sleep(cycles)
            case.call(source)
            graph.capture_end()
        return graph

    t.cuda.synchronize()
    t.cuda.empty_cache()
    start = t.cuda.mem_get_info()[0]
    first = late(cases[0], 400_000_000)
    done = t.cuda.Event()
    with t.cuda.stream(left):
        first.replay()
        done.record()
    del first
    second = late(cases[1], 0)
    running = not done.query()
    used = start - t.cuda.mem_get_info()[0]
    assert not running or used >= 2 * WeightGradient.bytes
    second.replay()
    t.cuda.synchronize()
    for case, w in zip(cases, want):
        assert t.equal(case.out, w)
