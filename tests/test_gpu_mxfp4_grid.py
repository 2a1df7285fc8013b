"""A grouped call whose tiles would be more than a grid has (needs an MI355X).  Codes are whole
numbers with one exponent: outputs are the formula's, rounded."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_mxfp4 import DEV, M, _check_guards, _gpu, guarded  # noqa: E402,F401
from test_gpu_mxfp4_limits import codes, packed, scales, values  # noqa: E402


def test_one_row_for_each_of_the_most_segments():
    n, d, n_seg, experts = 32768, 32, 65535, 2
    g = torch.Generator(device=DEV).manual_seed(1)
    stack, w = [], []
    for _ in range(experts):
        c, q = codes(g, n, d)
        stack.append(packed(q, n, d))
        w.append(values(c).double())
    stack = torch.stack(stack)
    xc, xq = codes(g, 7, d)
    each = torch.stack([(values(xc).double() @ v.T).bfloat16() for v in w])          # [expert][row of x][n]
    at = torch.arange(n_seg, device=DEV)
    se, ri, so = ((at % experts).int(), (at * 3 % 7).int(), torch.arange(n_seg + 1, device=DEV).int())
    y = guarded((n_seg, n), float("nan"), torch.bfloat16)
    qmm.qmm_mxfp4_grouped_gemm(stack, stack.shape[1], experts, n, d, xq, scales(7, d), 7, ri, se, so, n_seg, n_seg, 65, y)
    for r0 in range(0, n_seg, 4096):
        rows = slice(r0, min(r0 + 4096, n_seg))
        assert torch.equal(y[rows], each[se[rows].long(), ri[rows].long()]), r0
