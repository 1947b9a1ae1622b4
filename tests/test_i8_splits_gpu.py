"""8-bit integer products whose tiles are split over K: sums that meet in a cluster's shared memory
(up to eight splits of tiles that all run at once) or in the workspace (more of either)."""

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
