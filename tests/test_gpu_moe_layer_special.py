"""The expert layer's choice of logits and biases that are infinite, NaN, the types' largest or zeros of
either sign is the router's (needs an MI355X)."""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_moe_layer import DEV, F32, say  # noqa: E402
from test_gpu_moe_layer_choice import layer  # noqa: E402
from test_gpu_mxfp4 import _check_guards, _gpu  # noqa: E402,F401

SPECIAL = {"none": [], "masked": [-np.inf], "infinite": [np.inf, -np.inf], "largest": [3.3e38, -3.3e38, 0.0, -0.0],
           "nan": [np.nan, -np.inf], "all": [np.nan, np.inf, -np.inf, 3.3e38, -3.3e38, -0.0]}


@pytest.mark.parametrize("t", [1, 6, 16])
@pytest.mark.parametrize("ne,groups", [(8, 1), (64, 8), (100, 5), (128, 8), (160, 8), (256, 8), (256, 1), (300, 12), (512, 8),
                                       (1024, 16)])
def test_special_values(ne, groups, t):
    say("special", ne, groups, t)
    rng = np.random.default_rng(ne + groups + t)
    k = min(8, ne)
    topk, w = torch.empty(t, k, dtype=torch.int32, device=DEV), torch.empty(t, k, device=DEV)
    tables = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (ne, ne + 1, t * k, t * k)]
    ws = torch.empty(max(4, qmm.qmm_route_topk_workspace_bytes(t, ne)), dtype=torch.uint8, device=DEV)
    for score, bias, kind, renorm in itertools.product(["softmax", "sigmoid"], [None, "none", "largest", "all"], SPECIAL, [0, 1]):
        l = layer(t, ne, groups, score, bias is not None, score == "sigmoid", k, renorm, F32, rng)
        if SPECIAL[kind]:
            l.logits = np.where(rng.random((t, ne)) < 0.3, rng.choice(SPECIAL[kind], (t, ne)), l.logits)
        if bias is not None and SPECIAL[bias]:
            l.bias = np.where(rng.random(ne) < 0.1, rng.choice(SPECIAL[bias], ne), l.bias).astype(np.float32)
        i, o = l.inputs(), l.run()
        qmm.qmm_route_topk(i["logits"], F32, t, ne, i["ld"],
                           qmm.QMM_SCORE_SIGMOID if score == "sigmoid" else qmm.QMM_SCORE_SOFTMAX, i["bias"], groups, l.keep,
                           qmm.QMM_GROUP_TOP2 if l.top2 else qmm.QMM_GROUP_MAX, k, renorm, l.scale, topk, w, *tables, ws)
        what = score, bias, kind, renorm
        assert torch.equal(topk, o["topk"]), what
        assert torch.allclose(w, o["weights"], rtol=(ne + 64) * 2.0 ** -23, atol=0, equal_nan=True), what
        if kind in ("none", "masked", "largest") and bias is None:
            assert bool(torch.isfinite(o["out"].float()).all()), what
