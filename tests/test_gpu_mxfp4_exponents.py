"""Microscaled 4-bit products at the ends of the exponents' range (needs an MI355X).  Codes are whole
numbers and a call's exponents one on either side, so that a sum is a whole number times a power of two."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from oracle import mxfp4  # noqa: E402
from test_gpu_mxfp4 import M, _check_guards, _gpu, bf16_bits, dev, guarded, say  # noqa: E402,F401


@pytest.mark.parametrize("t", [1, 20, 50, 300])
@pytest.mark.parametrize("ex,ew", [(0, 254), (254, 0), (1, 253), (0, 130), (130, 0), (254, 100), (100, 254), (127, 127), (2, 140)])
def test_sums_are_exact(t, ex, ew):
    say("exponents", t, ex, ew)
    n, d = 130, 1056
    rng = np.random.default_rng(t + ex)
    whole = [0, 2, 4, 5, 6, 7, 10, 12, 15]
    wc, xc = rng.choice(whole, (n, d)), rng.choice(whole, (t, d))
    we = np.full((n, d // 32), ew, np.uint8)
    s = np.zeros((t, mxfp4.scale_bytes(d)), np.uint8)
    s[:, :d // 32] = ex
    wq, xq = mxfp4.pack_codes(wc), mxfp4.pack_codes(xc)
    packed = torch.empty(qmm.qmm_packed_bytes(M, n, d), dtype=torch.uint8, device="cuda")
    qmm.qmm_pack(M, n, d, dev(wq), dev(we), None, packed)
    y = guarded((t, n), float("nan"), torch.bfloat16)
    qmm.qmm_mxfp4_gemm(packed, t, n, d, dev(xq), dev(s), y, n)
    one = np.uint8(127)
    sums = mxfp4.dequant(xq, np.where(s, one, one)) @ mxfp4.dequant(wq, np.full_like(we, one)).T
    want = np.ldexp(sums, ex + ew - 254)
    assert 2.0 ** -124 <= np.abs(want[want != 0]).min() and np.abs(want).max() < 2.0 ** 127
    got = y.view(torch.int16).cpu().numpy().view(np.uint16)
    zero = want == 0                                           # of either sign
    assert np.array_equal(got[~zero], bf16_bits(want)[~zero]) and not np.any(got[zero] & 0x7FFF)
