"""8-bit integer products whose tiles are split over K: sums that meet in a cluster's shared memory
(up to eight splits of tiles that all run at once) or in the workspace (more of either)."""

import threading

import numpy as np
import pytest

import dense_fp32_gemm_row_gb300 as g
from tests.test_i8_gpu import operand, quiet, sums_of, t

pytestmark = pytest.mark.gpu


class Product:
    """One call, and what it has to give."""

    def __init__(self, T, N, K, splits, seed=0, algo="single"):
        self.shape, self.splits, self.algo = (T, N, K), splits, algo
        rng = np.random.default_rng(T + 3 * N + 7 * K + splits + 1000 * seed)
        (self.a, a, _), (self.b, b, _) = operand(rng, T, K), operand(rng, N, K)
        self.want = t().from_numpy(sums_of(a, b)).to(t().int32).cuda()
        self.out = t().full((T, N), -1, dtype=t().int32, device="cuda")

    def __call__(self, out=None, stream=None):
        return g.i8_matmul(self.a, self.b, dtype=t().int32, out=out, algo=self.algo, splits=self.splits,
                           stream=stream)

    def check(self):
        assert t().equal(self.out, self.want), (self.shape, self.splits)
        self.out.fill_(-1)
        t().cuda.synchronize()  # other streams do not wait for this one


# ---- in clusters --------------------------------------------------------------------------------


@pytest.mark.parametrize("splits", range(2, 9))
def test_clusters_of_every_size_back_to_back(splits):
    """Each call's sums overwrite stages that the calls around it fill: tokens and stages of all sorts."""
    cases = [Product(T, N, K, splits) for T, N, K in
             ((40, 200, 4096), (17, 128, 1100), (64, 640, 2048), (100, 300, 3000), (3, 1000, 8200), (16, 33, 5000))]
    made = [case() for _ in range(50) for case in cases]
    quiet()
    for i, y in enumerate(made):
        case = cases[i % len(cases)]
        assert t().equal(y, case.want), (case.shape, splits)


@pytest.mark.parametrize("splits", [2, 3, 4, 8])
def test_gated_clusters_back_to_back(splits):
    torch = t()
    rng = np.random.default_rng(splits)
    cases = []
    for T, N, K in ((40, 200, 4096), (100, 70, 3000), (9, 500, 2100)):
        a, b, c = (operand(rng, r, K)[0] for r in (T, N, N))
        for q in (b, c):
            q.scales.fill_(1e-4)
        cases.append((a, b, c, g.i8_gated(a, b, c, algo="single", splits=1)))
    made = [g.i8_gated(a, b, c, algo="single", splits=splits) for _ in range(40) for a, b, c, _ in cases]
    quiet()
    for i, h in enumerate(made):
        assert torch.equal(h, cases[i % len(cases)][3])


# ---- in the workspace: more splits than a cluster has CTAs, or than AUTO finds room for ---------------

WORKSPACE = ((40, 200, 4096, 12), (40, 200, 4096, 16), (3, 130, 9000, 9), (100, 300, 3000, 11), (64, 1000, 6000, 32),
             (17, 33, 40000, 256), (200, 129, 2600, 21))


def products(seed=0):
    return [Product(*case, seed=seed) for case in WORKSPACE]


def test_workspace_splits_back_to_back_with_every_other_form():
    torch = t()
    cases = products() + [Product(300, 20, 65540, 0, algo="auto"), Product(40, 200, 4096, 5), Product(300, 520, 1100, 0, algo="pair"),
                          Product(5, 700, 900, 0, algo="auto"), Product(600, 200, 300, 1)]
    order = np.random.default_rng(1).permutation(np.repeat(np.arange(len(cases)), 30))
    made = [cases[i]() for i in order]
    quiet()
    for i, y in zip(order, made):
        assert torch.equal(y, cases[i].want), (cases[i].shape, cases[i].splits)


def test_workspace_splits_of_gated_products():
    torch = t()
    rng = np.random.default_rng(2)
    for T, N, K, splits in WORKSPACE:
        a, b, c = (operand(rng, r, K)[0] for r in (T, N, N))
        for q in (b, c):
            q.scales.fill_(1e-4)
        for act in ("silu", "gelu"):
            want = g.i8_gated(a, b, c, act=act, algo="single", splits=1)
            made = [g.i8_gated(a, b, c, act=act, algo="single", splits=splits) for _ in range(10)]
            quiet()
            assert all(torch.equal(h, want) for h in made)


def test_workspace_splits_beside_the_other_operators_of_a_workspace():
    """Counters and partial sums of one stream's workspace, used in turn by kernels of three kinds."""
    torch = t()
    cases = products(3)
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = g.q8_store(torch.randn((65536, 256), generator=gen, device="cuda"))
    dy = torch.randn((65536, 256), generator=gen, device="cuda")
    a, b = torch.randn((256, 8192), generator=gen, device="cuda"), torch.randn((8192, 256), generator=gen, device="cuda")
    dw = g.q8_wgrad(q, dy)
    algos = (g.ALGO_FFMA, g.ALGO_3XTF32)
    want = [g.matmul(a, b, algo=algo, splits=8) for algo in algos]
    quiet()
    for _ in range(10):
        made, others = [], []
        for case in cases:
            made.append(case())
            others.append((dw, g.q8_wgrad(q, dy)))
            made.append(case())
            others += [(w, g.matmul(a, b, algo=algo, splits=8)) for w, algo in zip(want, algos)]
        quiet()
        for i, y in enumerate(made):
            assert torch.equal(y, cases[i // 2].want)
        assert all(torch.equal(x, y) for x, y in others)


def test_workspace_splits_on_two_streams():
    torch = t()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sides = [products(4), products(5)]
    torch.cuda.synchronize()
    made = []
    for _ in range(30):
        for cases in zip(*sides):
            for case, stream in zip(cases, streams):
                with torch.cuda.stream(stream):
                    made.append((case, case()))
    quiet()
    assert all(torch.equal(y, case.want) for case, y in made)


def test_workspace_splits_by_threads_at_once():
    torch = t()
    sides = [products(seed) for seed in (6, 7, 8)]
    torch.cuda.synchronize()
    made, errors = [[] for _ in sides], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(15):
                    made[i] += [(case, case()) for case in sides[i]]
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sides))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    quiet()
    assert not errors and all(torch.equal(y, case.want) for ms in made for case, y in ms)


# ---- workspace splits in graphs ------------------------------------------------------------------


def captured(cases, source):
    torch = t()
    torch.cuda.synchronize()
    for case in cases:  # the stream's workspace is there before the capture
        case(out=case.out, stream=source)
    torch.cuda.synchronize()
    for case in cases:
        case.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=source):
        for case in cases:
            case(out=case.out)
    return graph


def test_workspace_splits_in_two_graphs_of_one_stream():
    torch = t()
    source, left, right = (torch.cuda.Stream() for _ in range(3))
    sides = [products(9), products(10)]
    graphs = [captured(cases, source) for cases in sides]
    for _ in range(20):
        for _ in range(4):
            for graph, stream in zip(graphs, (left, right)):
                with torch.cuda.stream(stream):
                    graph.replay()
        quiet()
        for case in sides[0] + sides[1]:
            case.check()


def test_workspace_splits_in_a_graph_beside_calls_on_its_stream():
    torch = t()
    source, other = torch.cuda.Stream(), torch.cuda.Stream()
    cases, eager = products(11), products(12)
    graph = captured(cases, source)
    for _ in range(20):
        for _ in range(4):
            with torch.cuda.stream(other):
                graph.replay()
            for case in eager:
                case(out=case.out, stream=source)
        quiet()
        for case in cases + eager:
            case.check()


def test_a_captured_workspace_split_without_its_workspace():
    """Refused, and nothing of it in the graph; the capture goes on."""
    torch = t()
    case = Product(*WORKSPACE[0], seed=13)
    torch.cuda.synchronize()
    g.check(g.gemm_f32_release())
    source = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=source):
        with pytest.raises(g.GemmError) as e:
            case(out=case.out)
        case.out.fill_(7)
    assert e.value.status == g.ERR_CAPTURE
    graph.replay()
    quiet()
    assert bool((case.out == 7).all())
    again = captured([case], source)
    again.replay()
    quiet()
    case.check()
