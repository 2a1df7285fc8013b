"""Router on every way it chooses: a wave or a row of lanes a token, rounds or a
sort, one launch or two, groups of whole lanes or not (needs an MI355X)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
import test_gpu_fp8 as base  # noqa: E402
from test_gpu_fp8 import _check_guards, _gpu  # noqa: E402,F401

BF, F32 = qmm.QMM_BF16, qmm.QMM_F32

# t, experts, k, score, bias, groups, kept, two largest, renorm, dtype, pad
CASES = [(4, 129, 8, "sigmoid", True, 3, 2, True, True, BF, 0), (5, 130, 8, "softmax", False, 1, 1, False, True, F32, 1),
         (20, 256, 4, "sigmoid", True, 8, 4, True, True, F32, 0), (32, 256, 5, "sigmoid", False, 16, 3, False, False, BF, 0),
         (100, 256, 8, "sigmoid", True, 8, 4, True, True, F32, 3), (100, 256, 12, "softmax", True, 4, 2, False, True, F32, 0),
         (40, 200, 20, "sigmoid", True, 1, 1, False, True, F32, 0), (70, 250, 7, "softmax", False, 10, 4, True, True, BF, 2),
         (128, 100, 16, "sigmoid", False, 5, 3, True, True, F32, 0), (300, 130, 3, "softmax", False, 1, 1, False, True, F32, 0),
         (129, 256, 8, "softmax", False, 1, 1, False, False, BF, 0), (1000, 160, 6, "sigmoid", True, 8, 3, True, True, F32, 0),
         (17, 15, 15, "softmax", False, 1, 1, False, True, F32, 0), (200, 1, 1, "sigmoid", False, 1, 1, False, True, F32, 0),
         (200, 2, 2, "softmax", False, 2, 1, False, True, F32, 5), (5000, 144, 8, "sigmoid", True, 48, 20, True, True, BF, 0),
         (9000, 65, 9, "sigmoid", False, 13, 5, False, True, F32, 0), (140, 300, 8, "softmax", False, 12, 5, True, True, F32, 0)]


@pytest.mark.parametrize("case", CASES)
def test_route_variants(case):
    base.test_route_parity(case)


@pytest.mark.parametrize("t", [2, 10, 90, 600])
@pytest.mark.parametrize("ne,k", [(8, 3), (100, 8), (256, 8), (256, 16), (256, 40), (700, 6)])
def test_equal_values_go_to_the_lowest_experts(t, ne, k):
    l = np.zeros((t, ne))
    got = base.route(l, F32, ne, "sigmoid", None, 1, 1, False, k, True, 1.0)
    assert np.array_equal(got["topk"], np.tile(np.arange(k), (t, 1)))
    l[:, ne // 2:] = 1.0                                      # two values
    got = base.route(l, F32, ne, "softmax", None, 1, 1, False, k, True, 1.0)
    want = [(ne // 2 + j if j < ne - ne // 2 else j - (ne - ne // 2)) for j in range(k)]
    assert np.array_equal(got["topk"], np.tile(want, (t, 1)))


@pytest.mark.parametrize("t", [3, 12, 100, 700])
@pytest.mark.parametrize("ne", [40, 256, 512])
def test_fewer_experts_left_than_asked_for(t, ne):
    rng = np.random.default_rng(5000 + t + ne)
    l = np.full((t, ne), -np.inf)
    left = rng.integers(0, 9, t)
    want = np.full((t, 8), -1)
    for i, n in enumerate(left):
        e = rng.choice(ne, n, replace=False)
        l[i, e] = np.arange(n, 0, -1) - 100.0                 # e[0] is the largest
        want[i, :n] = e
    got = base.route(l, F32, ne, "softmax", None, 1, 1, False, 8, False, 1.0)
    assert np.array_equal(got["topk"], want)
    assert np.all(got["weights"][want < 0] == 0.0) and np.all(got["weights"][want >= 0] > 0.0)
    # 1 / (1 + e^-l) in fp32: e^92 is beyond its range, every one of these scores is 0
    # and equal, and the lower expert goes first
    got = base.route(l, F32, ne, "sigmoid", None, 1, 1, False, 8, False, 1.0)
    for i, n in enumerate(left):
        want[i, :n] = np.sort(want[i, :n])
    assert np.array_equal(got["topk"], want) and np.all(got["weights"] == 0.0)
