"""The expert layer's choice for every number of experts a lane (1, 2, 4, 8, 16), with one and two
tokens a wave, against the router's fp64 definition (needs an MI355X)."""
import functools

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_moe_layer import BF, DEV, F32, Layer, bf16_bits, say  # noqa: E402
from test_gpu_mxfp4 import _check_guards, _gpu  # noqa: E402,F401
from oracle import bf16_to_f64  # noqa: E402
import bit_weight_quantized_amd as qmm  # noqa: E402

# experts, groups: one; in whole lanes that exchange by DPP (2, 4, 8, 16 of a group); others, through LDS
SIZES = [(64, 1), (64, 8), (60, 5), (100, 1), (128, 1), (128, 32), (128, 8), (128, 4), (100, 10), (100, 50), (129, 1),
         (256, 1), (256, 32), (256, 16), (256, 8), (256, 4), (160, 8), (132, 33), (257, 1), (512, 1), (512, 8), (384, 24),
         (300, 12), (513, 1), (1024, 1), (1024, 8), (1024, 64), (700, 7)]


@functools.lru_cache(None)
def experts(ne):
    """A layer's weights, made once for every number of experts."""
    return Layer((1, ne, 1, 32, 32, "softmax", False, 1, 1, False, True, F32, 0, False), 7000 + ne)


def layer(t, ne, groups, score, bias, top2, k, renorm, dtype, rng):
    l = object.__new__(Layer)
    l.__dict__.update(experts(ne).__dict__)
    l.t, l.k, l.score, l.groups, l.keep, l.top2, l.renorm, l.dtype = t, k, score, groups, (groups + 1) // 2, top2, renorm, dtype
    l.ld_pad = 3 if bias else 0
    l.x = bf16_bits(rng.normal(0, 1, (t, 32)))
    # no two logits of a token closer than 2^-5 unless they are equal; equal ones among them
    l.logits = rng.integers(-100, 100, (t, ne)) / 32.0
    if dtype == BF:
        l.logits = bf16_to_f64(bf16_bits(l.logits))
    l.bias = (rng.integers(-8, 9, ne) / 32.0).astype(np.float32) if bias else None
    return l


@pytest.mark.parametrize("t", [1, 7, 8, 9, 16])
@pytest.mark.parametrize("ne,groups", SIZES)
def test_choice(ne, groups, t):
    say("choice", ne, groups, t)
    rng = np.random.default_rng(31 * ne + 7 * groups + t)
    keep = (groups + 1) // 2
    for n, (score, bias, top2, dtype) in enumerate([("softmax", False, False, F32), ("softmax", True, False, BF),
                                                    ("sigmoid", True, True, F32), ("sigmoid", False, False, BF),
                                                    ("softmax", False, True, F32)]):
        k = min([8, 1, 6, 16, 5][n], keep * (ne // groups))
        l = layer(t, ne, groups, score, bias, top2, k, n % 2 == 0, dtype, rng)
        # a probability with its bias, or two probabilities of a group, may come near another sum by
        # chance: such tokens are not compared (one of 8 with 1024 experts in 64 groups)
        l.check(l.run(), 0.5 if bias or top2 else 0.9)


@pytest.mark.parametrize("t", [3, 13])
@pytest.mark.parametrize("ne,groups", SIZES)
def test_equal_logits_go_to_the_lowest_experts(ne, groups, t):
    """Three values only: ties within a lane, between lanes and between groups."""
    rng = np.random.default_rng(ne + groups + t)
    for score, top2 in (("softmax", False), ("sigmoid", True)):
        l = layer(t, ne, groups, score, False, top2, min(16, (groups + 1) // 2 * (ne // groups)), True, F32, rng)
        l.logits = rng.choice([-1.0, 0.5, 1.25], (t, ne), p=[0.6, 0.37, 0.03])
        l.check(l.run(), 1.0)
        l.logits[:] = 0.25
        o = l.run()
        assert np.array_equal(o["topk"].cpu().numpy(), np.tile(np.arange(l.k), (t, 1)))
        l.check(o, 0.0)


@pytest.mark.parametrize("t", [2, 12])
@pytest.mark.parametrize("ne,groups", SIZES)
def test_masked_and_nan_logits(ne, groups, t):
    """Most experts masked, whole groups among them, fewer left than are asked for, or none."""
    rng = np.random.default_rng(3 * ne + groups + t)
    for score in ("softmax", "sigmoid"):
        l = layer(t, ne, groups, score, False, score == "sigmoid", min(8, ne), True, F32, rng)
        for i in range(t):
            left = rng.choice(ne, min(ne, 3 * i), replace=False)
            row = np.full(ne, -np.inf)
            row[left] = l.logits[i, left]
            l.logits[i] = row
        if score == "sigmoid":
            l.logits[t - 1, rng.integers(0, ne, 2)] = np.nan
        o = l.run()
        assert np.all(o["topk"].cpu().numpy()[0] == -1) and not o["weights"][0].any()
        l.check(o)


@pytest.mark.parametrize("ne,groups,t,k", [(256, 8, 1, 8), (256, 8, 16, 8), (160, 8, 9, 6), (128, 8, 16, 4), (512, 8, 5, 12),
                                           (1024, 16, 11, 16)])
def test_agrees_with_the_router(ne, groups, t, k):
    """The router's own choice of the same logits; weights to the order of fp32 sums."""
    rng = np.random.default_rng(ne + t)
    l = layer(t, ne, groups, "sigmoid", True, True, k, True, F32, rng)
    i, o = l.inputs(), l.run()
    topk, w = torch.empty(t, k, dtype=torch.int32, device=DEV), torch.empty(t, k, device=DEV)
    tables = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (ne, ne + 1, t * k, t * k)]
    ws = torch.empty(max(4, qmm.qmm_route_topk_workspace_bytes(t, ne)), dtype=torch.uint8, device=DEV)
    qmm.qmm_route_topk(i["logits"], F32, t, ne, i["ld"], qmm.QMM_SCORE_SIGMOID, i["bias"], groups, l.keep, qmm.QMM_GROUP_TOP2, k,
                       True, l.scale, topk, w, *tables, ws)
    assert torch.equal(topk, o["topk"])
    assert torch.allclose(w, o["weights"], rtol=(k + 4) * 2.0 ** -23, atol=0)
