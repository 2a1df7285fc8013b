"""Host refusals of the microscaled 4-bit path: every call here fails validation before any
HIP call, or is a no-op."""
import os

import pytest

import bit_weight_quantized_amd as qmm

pytestmark = pytest.mark.skipif(not os.path.exists(qmm.lib_path()),
                                reason="libqmm.so not built (run __graft_entry__.build())")

E_ARG, E_SHAPE, E_ALIGN, E_UNSUPPORTED, E_WS = 1, 2, 3, 4, 5
P = 1 << 20          # an aligned fake device address: validation never dereferences it


def expect(status, fn, *args):
    with pytest.raises(qmm.QmmError) as ei:
        fn(*args, stream=0)
    assert ei.value.status == status, (ei.value, qmm.qmm_last_error())
    assert qmm.qmm_last_error()


def changer(good):
    def with_(*pairs):
        a = list(good)
        for i, v in zip(pairs[0::2], pairs[1::2]):
            a[i] = v
        return a
    return with_


def test_scale_bytes():
    assert [qmm.qmm_mxfp4_scale_bytes(d) for d in (32, 512, 544, 5120, 65536)] == [16, 16, 32, 160, 2048]
    assert [qmm.qmm_mxfp4_scale_bytes(d) for d in (0, -32, 16, 33, 65568)] == [0] * 5


def test_quant_refusals():
    f = qmm.qmm_mxfp4_quant                     # x, t, d, ldx, rule, q, scales
    with_ = changer([P, 4, 128, 128, 0, P, P])
    expect(E_ARG, f, *with_(1, -1))
    expect(E_ARG, f, *with_(2, 0))
    expect(E_SHAPE, f, *with_(2, 48, 3, 48))
    expect(E_SHAPE, f, *with_(2, 65568, 3, 65568))
    expect(E_SHAPE, f, *with_(1, (1 << 24) + 1))
    expect(E_ARG, f, *with_(3, 120))
    expect(E_ARG, f, *with_(4, 2))
    expect(E_ARG, f, *with_(4, -1))
    expect(E_ALIGN, f, *with_(3, 132))
    for i in (0, 5, 6):
        expect(E_ARG, f, *with_(i, None))
        expect(E_ALIGN, f, *with_(i, P + 8))
    f(None, 0, 128, 128, 0, None, None, stream=0)


def test_gemm_refusals():
    f = qmm.qmm_mxfp4_gemm                      # packed, t, n, d, x, xs, y, ldy
    with_ = changer([P, 4, 32, 128, P, P, P, 32])
    for i in (0, 4, 5, 6):
        expect(E_ARG, f, *with_(i, None))
    expect(E_ARG, f, *with_(1, -1))
    expect(E_SHAPE, f, *with_(1, (1 << 24) + 1))
    expect(E_ARG, f, *with_(2, 0))
    expect(E_SHAPE, f, *with_(2, (1 << 28) + 1, 7, 1 << 30))
    expect(E_SHAPE, f, *with_(2, 1 << 17, 3, 32768, 7, 1 << 17))    # 2 GiB of codes
    expect(E_SHAPE, f, *with_(3, 80))
    expect(E_SHAPE, f, *with_(3, 65568))
    expect(E_ARG, f, *with_(7, 31))
    expect(E_ALIGN, f, *with_(0, P + 128))
    expect(E_ALIGN, f, *with_(4, P + 8))
    expect(E_ALIGN, f, *with_(5, P + 8))
    expect(E_ALIGN, f, *with_(6, P + 1))
    f(*with_(1, 0), stream=0)


@pytest.mark.parametrize("glu", [False, True])
def test_grouped_refusals(glu):
    f = qmm.qmm_mxfp4_grouped_gemm_swiglu if glu else qmm.qmm_mxfp4_grouped_gemm
    size = qmm.qmm_packed_bytes(qmm.QMM_MXFP4_G32, 64, 128)
    # packed, stride, n_experts, n, d, x, xs, t_x, row_index, seg_expert, seg_offsets, n_seg, m_total, most, (rule, h, hq, hs) y
    with_ = changer([P, size, 2, 64, 128, P, P, 4, P, P, P, 1, 4, 4] + ([0, None, P, P] if glu else [P]))
    for i in (0, 5, 6, 9, 10):
        expect(E_ARG, f, *with_(i, None))
    expect(E_ARG, f, *with_(1, size - 256))
    expect(E_ARG, f, *with_(1, size + 128))
    expect(E_ARG, f, *with_(2, 0))
    expect(E_ARG, f, *with_(3, 0))
    expect(E_SHAPE, f, *with_(4, 72))
    expect(E_ARG, f, *with_(7, 0))
    expect(E_SHAPE, f, *with_(7, 1 << 25))
    expect(E_SHAPE, f, *with_(4, 512, 1, 1 << 20, 7, 1 << 23))     # codes of x of 2 GiB
    expect(E_ARG, f, *with_(11, -1))
    expect(E_SHAPE, f, *with_(11, 65536))
    expect(E_ARG, f, *with_(12, -1))
    expect(E_ARG, f, *with_(13, 0))
    expect(E_ALIGN, f, *with_(0, P + 16))
    for i in (5, 6):
        expect(E_ALIGN, f, *with_(i, P + 8))
    for i in (8, 9, 10):
        expect(E_ALIGN, f, *with_(i, P + 2))
    if glu:
        expect(E_SHAPE, f, *with_(3, 63, 15, P, 16, None, 17, None))
        expect(E_SHAPE, f, *with_(3, 48))                          # 24 outputs are not whole blocks
        expect(E_ARG, f, *with_(14, 2))
        expect(E_ARG, f, *with_(15, P))                            # both forms
        expect(E_ARG, f, *with_(16, None))                         # hs without hq
        expect(E_ARG, f, *with_(17, None))
        expect(E_ARG, f, *with_(16, None, 17, None))               # none
        expect(E_ALIGN, f, *with_(15, P + 1, 16, None, 17, None))
        expect(E_ALIGN, f, *with_(16, P + 8))
        expect(E_ALIGN, f, *with_(17, P + 8))
    else:
        expect(E_ARG, f, *with_(14, None))
        expect(E_ALIGN, f, *with_(14, P + 1))
    f(*with_(11, 0), stream=0)
    f(*with_(12, 0), stream=0)


def test_moe_layer_workspace():
    f = qmm.qmm_moe_layer_workspace_bytes
    assert f(1, 8, 2048) == 4 * 8 * 2048 and f(16, 16, 32) == 4 * 256 * 32
    assert [f(0, 1, 32), f(17, 1, 32), f(1, 65, 32), f(16, 17, 32), f(1, 0, 32), f(1, 1, 33), f(1, 1, 65568)] == [0] * 7


def test_moe_layer_refusals():
    f = qmm.qmm_moe_layer
    d, inter, ne, t, k = 128, 64, 8, 4, 2
    gu, dn = qmm.qmm_packed_bytes(qmm.QMM_MXFP4_G32, 2 * inter, d), qmm.qmm_packed_bytes(qmm.QMM_MXFP4_G32, d, inter)
    # 0 fmt, 1 gate_up, 2 stride, 3 down, 4 stride, 5 n_experts, 6 d, 7 inter, 8 x, 9 t, 10 logits, 11 dtype, 12 ld,
    # 13 score, 14 bias, 15 n_groups, 16 keep, 17 group score, 18 k, 19 renorm, 20 scale, 21 shared, 22 topk,
    # 23 weights, 24 out, 25 ws
    class Ws:
        def __init__(self, at, n):
            self.at, self.n = at, n

        def data_ptr(self):
            return self.at

        def numel(self):
            return self.n

        def element_size(self):
            return 1
    need = qmm.qmm_moe_layer_workspace_bytes(t, k, inter)
    with_ = changer([qmm.QMM_MXFP4_G32, P, gu, P, dn, ne, d, inter, P, t, P, qmm.QMM_F32, ne, 0, None, 1, 1, 0, k, 1, 1.0,
                     None, P, P, P, Ws(P, need)])
    expect(E_UNSUPPORTED, f, *with_(0, qmm.QMM_AFFINE4_G64))
    expect(E_ARG, f, *with_(0, 7))
    for i in (1, 3, 8, 10, 22, 23, 24):
        expect(E_ARG, f, *with_(i, None))
    expect(E_ARG, f, *with_(2, gu - 256))
    expect(E_ARG, f, *with_(2, gu + 64))
    expect(E_ARG, f, *with_(4, dn - 256))
    expect(E_ARG, f, *with_(4, dn + 64))
    expect(E_ARG, f, *with_(5, 0))
    expect(E_SHAPE, f, *with_(5, 1025, 12, 1025))
    for i in (6, 7):
        expect(E_ARG, f, *with_(i, 0))
        expect(E_SHAPE, f, *with_(i, 48))
        expect(E_SHAPE, f, *with_(i, 65568))
    expect(E_SHAPE, f, *with_(6, 65536, 7, 65536))            # 4 GiB of codes
    expect(E_ARG, f, *with_(9, -1))
    expect(E_SHAPE, f, *with_(9, 17))
    expect(E_SHAPE, f, *with_(9, 16, 18, 17, 5, 32, 12, 32))  # 272 pairs
    expect(E_ARG, f, *with_(11, 3))
    expect(E_ARG, f, *with_(12, ne - 1))
    expect(E_ARG, f, *with_(13, 2))
    expect(E_SHAPE, f, *with_(15, 3))
    expect(E_SHAPE, f, *with_(15, 0))
    expect(E_ARG, f, *with_(15, 4, 16, 5))
    expect(E_ARG, f, *with_(16, 0))
    expect(E_ARG, f, *with_(17, 2))
    expect(E_ARG, f, *with_(18, 0))
    expect(E_SHAPE, f, *with_(18, 9))
    expect(E_SHAPE, f, *with_(18, 65, 5, 128, 12, 128, 9, 1))
    expect(E_ARG, f, *with_(20, float("inf")))
    expect(E_ARG, f, *with_(20, float("nan")))
    for i, off in ((1, 128), (3, 128), (8, 8), (10, 2), (14, 2), (21, 4), (22, 2), (23, 2), (24, 4)):
        expect(E_ALIGN, f, *with_(i, P + off))
    expect(E_WS, f, *with_(25, None))
    expect(E_WS, f, *with_(25, Ws(P, need - 1)))
    expect(E_ALIGN, f, *with_(25, Ws(P + 8, need)))
    f(*with_(9, 0, 1, None, 8, None, 25, None), stream=0)
