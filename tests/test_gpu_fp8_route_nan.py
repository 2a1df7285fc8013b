"""NaN and infinite logits under each way in which the router ranks (needs an MI355X)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
import test_gpu_fp8 as base  # noqa: E402
from test_gpu_fp8 import _check_guards, _gpu  # noqa: E402,F401


# one launch by rows and by waves, two launches, more than 256 experts
@pytest.mark.parametrize("t,ne", [(3, 16), (3, 160), (9, 160), (70, 256), (300, 64), (6, 400)])
@pytest.mark.parametrize("bias,top2", [(False, False), (True, False), (False, True)])
def test_softmax_with_a_nan(t, ne, bias, top2):
    """Where c is the logit the others are chosen, their weights NaN; where c is made
    from p every c of the token is NaN and nothing is chosen.  Other tokens are untouched."""
    rng = np.random.default_rng(9900 + t + ne)
    l = rng.integers(-200, 200, (t, ne)) / 64.0
    l[1, 3] = np.nan
    groups, keep, k = (4, 4, 3) if top2 else (1, 1, 3)
    b = np.zeros(ne, np.float32) if bias else None
    got = base.route(l, qmm.QMM_F32, ne, "softmax", b, groups, keep, top2, k, True, 1.0)
    clean = l.copy()
    clean[1, 3] = -np.inf
    want = base.route(clean, qmm.QMM_F32, ne, "softmax", b, groups, keep, top2, k, True, 1.0)
    other = np.arange(t) != 1
    assert np.array_equal(got["topk"][other], want["topk"][other])
    assert np.array_equal(got["weights"][other], want["weights"][other])
    if bias or top2:
        assert np.all(got["topk"][1] == -1) and np.all(got["weights"][1] == 0.0) and np.all(got["slot_row"][1] == -1)
    else:
        assert np.array_equal(got["topk"][1], want["topk"][1]) and np.isnan(got["weights"][1]).all()
    offsets, rows, slot = base.tables_fast(got["topk"], ne)
    assert np.array_equal(got["seg_offsets"], offsets) and np.array_equal(got["row_index"], rows)
    assert np.array_equal(got["slot_row"], slot)
