"""Host refusals of the block-scaled e4m3 path, the top-k router, the gather and
the norms: every call here fails validation before any HIP call, or is a no-op."""
import os

import pytest

import bit_weight_quantized_amd as qmm

pytestmark = pytest.mark.skipif(not os.path.exists(qmm.lib_path()),
                                reason="libqmm.so not built (run __graft_entry__.build())")

E_ARG, E_SHAPE, E_ALIGN, E_WS = 1, 2, 3, 5
P = 1 << 20          # an aligned fake device address: validation never dereferences it
BF, F32 = qmm.QMM_BF16, qmm.QMM_F32


def expect(status, fn, *args):
    with pytest.raises(qmm.QmmError) as ei:
        fn(*args, stream=0)
    assert ei.value.status == status, (ei.value, qmm.qmm_last_error())
    assert qmm.qmm_last_error()


def test_quant_refusals():
    f = qmm.qmm_fp8_quant                       # x, t, d, ldx, q, scales
    expect(E_ARG, f, P, -1, 128, 128, P, P)
    expect(E_ARG, f, P, 4, 0, 128, P, P)
    expect(E_SHAPE, f, P, 4, 24, 24, P, P)      # d % 16
    expect(E_SHAPE, f, P, 4, 65552, 65552, P, P)
    expect(E_SHAPE, f, P, (1 << 24) + 1, 16, 16, P, P)
    expect(E_SHAPE, f, P, 1 << 20, 65536, 65536, P, P)   # t·nb > 2^28
    expect(E_ARG, f, P, 4, 128, 127, P, P)      # ldx < d
    expect(E_ALIGN, f, P, 4, 128, 132, P, P)    # ldx % 8
    expect(E_ALIGN, f, P + 8, 4, 128, 128, P, P)
    expect(E_ALIGN, f, P, 4, 128, 128, P + 8, P)
    expect(E_ALIGN, f, P, 4, 128, 128, P, P + 2)
    for i in (0, 4, 5):
        a = [P, 4, 128, 128, P, P]
        a[i] = None
        expect(E_ARG, f, *a)
    f(None, 0, 128, 128, None, None, stream=0)  # no rows: nothing to do


def test_gemm_refusals():
    f = qmm.qmm_fp8_gemm                        # w, ws, t, n, d, x, xs, y, ldy
    good = [P, P, 4, 32, 128, P, P, P, 32]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return a
    for i in (0, 1, 5, 6, 7):
        expect(E_ARG, f, *with_(i, None))
    expect(E_ARG, f, *with_(2, -1))
    expect(E_SHAPE, f, *with_(2, (1 << 24) + 1))
    expect(E_ARG, f, *with_(3, 0))
    expect(E_SHAPE, f, *with_(3, (1 << 28) + 1))
    expect(E_SHAPE, f, *with_(4, 120))
    expect(E_SHAPE, f, *with_(4, 65552))
    expect(E_ARG, f, *with_(8, 31))
    expect(E_ALIGN, f, *with_(0, P + 8))
    expect(E_ALIGN, f, *with_(5, P + 8))
    expect(E_ALIGN, f, *with_(1, P + 2))
    expect(E_ALIGN, f, *with_(6, P + 2))
    expect(E_ALIGN, f, *with_(7, P + 1))
    f(*with_(2, 0), stream=0)


@pytest.mark.parametrize("name", ["qmm_fp8_grouped_gemm", "qmm_fp8_grouped_gemm_swiglu"])
def test_grouped_refusals(name):
    f = getattr(qmm, name)
    # w, ws, n_experts, n, d, x, xs, t_x, row_index, seg_expert, seg_offsets, n_seg, m_total, max_seg_rows, y
    good = [P, P, 2, 32, 128, P, P, 4, P, P, P, 1, 4, 4, P]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return a
    for i in (0, 1, 5, 6, 9, 10, 14):
        expect(E_ARG, f, *with_(i, None))
    expect(E_ARG, f, *with_(2, 0))
    expect(E_SHAPE, f, *with_(4, 72))
    expect(E_ARG, f, *with_(7, 0))
    expect(E_SHAPE, f, *with_(7, 1 << 24))      # x of 2 GiB
    expect(E_ARG, f, *with_(11, -1))
    expect(E_SHAPE, f, *with_(11, 65536))
    expect(E_ARG, f, *with_(12, -1))
    expect(E_ARG, f, *with_(13, 0))
    for i in (0, 5):
        expect(E_ALIGN, f, *with_(i, P + 8))
    for i in (1, 6, 8, 9, 10):
        expect(E_ALIGN, f, *with_(i, P + 2))
    expect(E_ALIGN, f, *with_(14, P + 1))
    if name.endswith("swiglu"):
        expect(E_SHAPE, f, *with_(3, 31))
    f(*with_(11, 0), stream=0)                  # no segments, no rows: nothing to do
    f(*with_(12, 0), stream=0)


def test_route_refusals():
    f = qmm.qmm_route_topk
    # logits, dtype, t, ne, ld, score, bias, groups, keep, by, k, renorm, scale, topk, w, se, so, ri, sr, ws
    good = [P, F32, 4, 64, 64, 1, P, 8, 4, 1, 6, True, 1.0, P, P, P, P, P, P, None]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return a
    for i in (0, 13, 14, 15, 16, 17, 18):
        expect(E_ARG, f, *with_(i, None))
    for i, v in ((1, 3), (1, 0), (2, -1), (3, 0), (4, 63), (5, 2), (8, 0), (8, 9), (9, 2), (10, 0),
                 (12, float("inf")), (12, float("nan"))):
        expect(E_ARG, f, *with_(i, v))
    for i, v in ((7, 0), (7, 7), (7, 128), (10, 65), (2, 1 << 25)):
        expect(E_SHAPE, f, *with_(i, v))
    expect(E_SHAPE, f, P, F32, 4, 1025, 1025, 1, None, 1, 1, 0, 6, True, 1.0, P, P, P, P, P, P, None)
    expect(E_SHAPE, f, P, F32, 4, 4, 4, 1, None, 1, 1, 0, 5, True, 1.0, P, P, P, P, P, P, None)
    for i in (0, 6, 13, 14, 15, 16, 17, 18):
        expect(E_ALIGN, f, *with_(i, P + 2))
    expect(E_ALIGN, f, *with_(0, P + 1))
    expect(E_WS, f, *with_(2, 129))             # more than 128 tokens take a workspace


def test_route_workspace():
    w = qmm.qmm_route_topk_workspace_bytes
    assert w(1, 256) == w(128, 256) == w(0, 256) == w(-1, 4) == w(200, 1025) == w(200, 0) == 0
    for t in (129, 1000, 8192, 8193, 16384, 32769, 100000, 1 << 24):
        for ne in (1, 60, 1024):
            assert 0 < w(t, ne) <= 4 * ne * -(-t // 32) and w(t, ne) <= 4 * ne * 256


def test_gather_refusals():
    f = qmm.qmm_moe_gather                      # o, m_total, d, t, k, slot_row, weights, shared, out
    good = [P, 8, 64, 4, 2, P, P, P, P]

    def with_(i, v):
        a = list(good)
        a[i] = v
        return a
    for i in (0, 5, 6, 8):
        expect(E_ARG, f, *with_(i, None))
    for i in (1, 3):
        expect(E_ARG, f, *with_(i, -1))
    expect(E_ARG, f, *with_(4, 0))
    expect(E_SHAPE, f, *with_(4, 65))
    expect(E_SHAPE, f, *with_(2, 60))
    expect(E_SHAPE, f, *with_(2, 65544))
    for i in (0, 7, 8):
        expect(E_ALIGN, f, *with_(i, P + 8))
    for i in (5, 6):
        expect(E_ALIGN, f, *with_(i, P + 2))
    f(*with_(3, 0), stream=0)


def test_norm_refusals():
    f = qmm.qmm_norm_residual
    # t, d, o, ldo, post, gate, ldg, gate_rows, r, type, ldr, scale, r_out, ldr_out, pre, offset, eps, h, ldh, q, qs
    good = [4, 64, P, 64, P, P, 64, 1, P, BF, 64, 1.0, P, 64, P, 0.0, 1e-6, P, 64, P, P]

    def with_(*iv):
        a = list(good)
        for i, v in zip(iv[::2], iv[1::2]):
            a[i] = v
        return a
    for iv in ((0, -1), (1, 0), (9, 0), (8, None), (2, None), (14, None), (19, None), (20, None), (3, 63), (10, 63),
               (13, 63), (18, 63), (6, 63), (7, 0), (16, -1.0), (16, float("nan")), (11, float("inf")),
               (15, float("nan")), (12, None, 17, None, 19, None, 20, None)):
        expect(E_ARG, f, *with_(*iv))
    for iv in ((1, 60), (1, 65544), (0, (1 << 24) + 1)):
        expect(E_SHAPE, f, *with_(*iv))
    for i in (2, 4, 5, 8, 12, 14, 17):
        expect(E_ALIGN, f, *with_(i, P + 8))
    for i in (3, 6, 10, 13, 18):
        expect(E_ALIGN, f, *with_(i, 68))
    expect(E_ALIGN, f, *with_(19, P + 4))
    expect(E_ALIGN, f, *with_(20, P + 2))
    f(*with_(0, 0), stream=0)
