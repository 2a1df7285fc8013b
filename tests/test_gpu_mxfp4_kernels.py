"""Every kernel of the microscaled 4-bit path by a shape of its own (needs an MI355X)."""
import numpy as np
import pytest

import mxfp4_shapes as S
import test_gpu_mxfp4 as T
from oracle import mxfp4

pytestmark = pytest.mark.gpu
_gpu, _check_guards = T._gpu, T._check_guards


@pytest.mark.parametrize("t,n,d", [*S.DENSE_ROWS.values(), *S.DENSE_64, *S.DENSE_256])
def test_dense(t, n, d):
    T.test_gemm(t, n, d)


@pytest.mark.parametrize("n,d,lengths", [s for (_, _, g), s in S.GROUPED_ROWS.items() if not g] + S.GROUPED_64 + S.GROUPED_256)
def test_grouped(n, d, lengths):
    T.test_grouped(n, d, lengths, True)


@pytest.mark.parametrize("fit", [None, True])
@pytest.mark.parametrize("n,d,lengths", [s for (_, _, g), s in S.GROUPED_ROWS.items() if g] + S.GROUPED_64 + S.GROUPED_256)
def test_grouped_swiglu(n, d, lengths, fit):
    T.test_grouped_swiglu(n, d, lengths, fit)


@pytest.mark.parametrize("t,n,d", [(40, 640, 5120), (300, 1024, 5120), (1100, 4096, 2080)])
def test_rows_do_not_depend_on_each_other(t, n, d):
    """Rows repeated in another order give the same bits wherever they lie: nothing leaks between rows or tiles."""
    rng = np.random.default_rng(5)
    _, packed = T.weights(rng, n, d)
    q, s = T.rows(rng, 7, d)
    order = rng.integers(0, 7, t)
    y = T.guarded((t, n), float("nan"), T.torch.bfloat16)
    T.qmm.qmm_mxfp4_gemm(packed, t, n, d, T.dev(q[order]), T.dev(s[order]), y, n)
    got = y.view(T.torch.int16).cpu().numpy()
    for i in range(7):
        rows = got[order == i]
        assert np.all(rows == rows[0])


def test_a_row_of_zeros_and_a_row_of_the_largest_codes():
    t, n, d = 2, 96, 544
    rng = np.random.default_rng(6)
    w, packed = T.weights(rng, n, d)
    q, s = T.rows(rng, t, d)
    q[0], s[0] = 0, 0
    q[1] = 0x77
    y = T.guarded((t, n), float("nan"), T.torch.bfloat16)
    T.qmm.qmm_mxfp4_gemm(packed, t, n, d, T.dev(q), T.dev(s), y, n)
    got = T.as_f64(y)
    ref, rest = mxfp4.gemm(mxfp4.dequant(q, s), w)
    assert np.all(got[0] == 0) and np.all(np.abs(got - ref) <= mxfp4.gemm_tolerance(ref, rest))
