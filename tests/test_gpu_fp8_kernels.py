"""GPU parity of the block-scaled products and the norms on every kernel they choose
from, by the shapes of tests/fp8_shapes.py (needs an MI355X).  Tolerances:
oracle/fp8.py."""
import numpy as np
import pytest

from oracle import fp8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
import fp8_shapes as S  # noqa: E402
import test_gpu_fp8 as base  # noqa: E402
from test_gpu_fp8 import (_check_guards, _gpu, as_f64, codes, dense, dev, guarded, say,  # noqa: E402,F401
                          scales, segments)

BF, F32 = qmm.QMM_BF16, qmm.QMM_F32
GROUPED = list(S.GROUPED_ROWS.values()) + S.GROUPED_64 + S.GROUPED_256


@pytest.mark.parametrize("t,n,d", list(S.DENSE_ROWS.values()) + S.DENSE_64 + S.DENSE_256)
def test_dense(t, n, d):
    say("dense", t, n, d)
    y, ref, tol = dense(t, n, d, 9000 + t + n + d)
    assert np.all(np.abs(y - ref) <= tol)


def routed(n, d, lengths, seed, swiglu):
    """Outputs and their references by segment; some rows and an expert do not exist."""
    rng = np.random.default_rng(seed)
    ne, m, t_x, nb, sb = 5, sum(lengths), 211, fp8.blocks(d), fp8.blocks(n // 2)
    experts, offs, rows = segments(rng, lengths, ne, t_x)
    rows[::37] = t_x
    experts[len(lengths) // 2] = -1
    w = codes(rng, ne, n, d)
    ws = scales(rng, ne, 2 * sb if swiglu else fp8.blocks(n), nb) * np.float32(0.002 if swiglu else 1.0)
    x, xs = codes(rng, t_x, d), scales(rng, t_x, nb) * np.float32(0.1 if swiglu else 1.0)
    y = guarded((m, n // 2 if swiglu else n), 0.0, torch.bfloat16)
    f = qmm.qmm_fp8_grouped_gemm_swiglu if swiglu else qmm.qmm_fp8_grouped_gemm
    f(dev(w), dev(ws), ne, n, d, dev(x), dev(xs), t_x, dev(rows), dev(experts), dev(offs), len(lengths), m, max(lengths), y)
    y = as_f64(y.view(torch.int16))
    bad = (rows == t_x) | np.repeat(experts < 0, lengths)
    assert np.isnan(y[bad]).all()
    rows = np.where(rows == t_x, 0, rows)
    for i, e in enumerate(experts):
        at = slice(offs[i], offs[i + 1])
        if e < 0 or not lengths[i]:
            continue
        if swiglu:
            nh = n // 2
            g, rg = fp8.gemm(x[rows[at]], xs[rows[at]], w[e, :nh], ws[e, :sb])
            u, ru = fp8.gemm(x[rows[at]], xs[rows[at]], w[e, nh:], ws[e, sb:])
            ref, tol = fp8.swiglu_tolerance(g, u, rg, ru)
        else:
            ref, rest = fp8.gemm(x[rows[at]], xs[rows[at]], w[e], ws[e])
            tol = fp8.gemm_tolerance(ref, rest)
        ok = np.abs(y[at] - ref) <= tol
        assert np.all(ok | bad[at][:, None]), (i, lengths[i])


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("n,d,lengths", GROUPED)
def test_grouped(n, d, lengths, swiglu):
    say("grouped", n, d, len(lengths), swiglu)
    routed(n, d, lengths, 9500 + n, swiglu)


@pytest.mark.parametrize("rt", [BF, F32])
@pytest.mark.parametrize("t,d", list(S.NORMS.values()))
def test_norm(t, d, rt):
    # tokens, width, residual type, post weights, gate rows, block output, offset, h, codes, in place
    base.test_norm_parity((t, d, rt, True, 2, True, 1.0, True, True, False))


@pytest.mark.parametrize("t,d", list(S.NORMS.values()))
def test_norm_without_a_block_output(t, d):
    base.test_norm_parity((t, d, BF, False, 0, False, 0.0, True, True, True))
