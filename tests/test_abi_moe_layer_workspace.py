"""Sizes of the expert layer's workspace that the call takes and refuses.  Sizes that it takes
are shown by the refusal that follows the size's, of an address that is not aligned: no call
here gets as far as a launch."""
import os

import pytest

import bit_weight_quantized_amd as qmm
from test_abi_mxfp4 import E_ALIGN, E_WS, P, expect

pytestmark = pytest.mark.skipif(not os.path.exists(qmm.lib_path()),
                                reason="libqmm.so not built (run __graft_entry__.build())")


class Ws:
    def __init__(self, at, n):
        self.at, self.n = at, n

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def element_size(self):
        return 1


@pytest.mark.parametrize("t,ne,k,d,inter", [(1, 256, 8, 3584, 2048), (4, 8, 2, 128, 64), (7, 60, 4, 2080, 1056), (1, 1, 1, 32, 32)])
def test_the_whole_workspace_and_half_of_it(t, ne, k, d, inter):
    gu, dn = (qmm.qmm_packed_bytes(qmm.QMM_MXFP4_G32, *s) for s in ((2 * inter, d), (d, inter)))

    def args(ws):
        return (qmm.QMM_MXFP4_G32, P, gu, P, dn, ne, d, inter, P, t, P, qmm.QMM_F32, ne, 0, None, 1, 1, 0, k, 1, 1.0, None, P, P,
                P, ws)
    need = qmm.qmm_moe_layer_workspace_bytes(t, k, inter)
    half = 2 * t * k * inter
    assert need == 2 * half
    for size in (half, half + 16, need - 16, need, need + 1, need + 256):
        expect(E_ALIGN, qmm.qmm_moe_layer, *args(Ws(P + 8, size)))
    for size in (0, 16, half - 16, half - 1, half + 1, half + 8, need - 1):
        expect(E_WS, qmm.qmm_moe_layer, *args(Ws(P, size)))
    expect(E_WS, qmm.qmm_moe_layer, *args(None))
