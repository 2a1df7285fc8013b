"""SwiGLU whose outputs end inside a block of columns, by every kernel (needs an MI355X)."""
import pytest

import test_gpu_mxfp4 as T
from mxfp4_ragged_shapes import RAGGED

pytestmark = pytest.mark.gpu
_gpu, _check_guards = T._gpu, T._check_guards


@pytest.mark.parametrize("n,d,lengths", [s for _, s in RAGGED])
def test_swiglu_of_ragged_widths(n, d, lengths):
    T.test_grouped_swiglu(n, d, lengths, None)
