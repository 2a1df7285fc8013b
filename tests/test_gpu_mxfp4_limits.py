"""The microscaled 4-bit calls and the expert layer at the ends of their ranges: the most rows,
the widest and the longest matrices, stacks past 4 GiB (needs an MI355X).  Codes are whole
numbers with one exponent, so that every sum is exact and outputs are the formula's, rounded."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_moe_layer import Layer  # noqa: E402
from test_gpu_mxfp4 import DEV, M, _check_guards, _gpu, guarded, say  # noqa: E402,F401

F32 = qmm.QMM_F32
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
WHOLE = torch.tensor([0, 2, 4, 5, 10, 12], dtype=torch.uint8)          # 0, 1, 2, 3, -1, -2


def codes(g, rows, d):
    c = WHOLE.to(DEV)[torch.randint(0, len(WHOLE), (rows, d), generator=g, device=DEV)]
    return c, (c[:, 0::2] | c[:, 1::2] << 4).contiguous()


def values(c):
    return VALUES.to(DEV)[c.long()]


def repeated(rows, n):
    """n rows, the given ones over and over (indexing gives zeros for rows past 2^30 bytes)."""
    out = rows.repeat(-(-n // rows.shape[0]), 1)[:n].contiguous()
    at = torch.arange(max(0, n - 999), n, device=DEV)
    assert torch.equal(out[-at.numel():], rows[at % rows.shape[0]])
    return out


def scales(rows, d):
    s = torch.zeros(rows, qmm.qmm_mxfp4_scale_bytes(d), dtype=torch.uint8, device=DEV)
    s[:, :d // 32] = 127
    return s


def packed(c, n, d):
    blob = torch.empty(qmm.qmm_packed_bytes(M, n, d), dtype=torch.uint8, device=DEV)
    qmm.qmm_pack(M, n, d, c, torch.full((n, d // 32), 127, dtype=torch.uint8, device=DEV), None, blob)
    return blob


# the most rows; the most weight rows a call of 32 codes takes, few rows and a tile; the longest reductions
@pytest.mark.parametrize("t,n,d", [(1 << 24, 8, 32), (1 << 24, 300, 32), (1, (1 << 27) - 48, 32), (200, (1 << 22) + 5, 64),
                                   (1, 33, 65536), (70, 130, 65504), (300, 300, 65536)])
def test_gemm(t, n, d):
    say("limits", t, n, d)
    g = torch.Generator(device=DEV).manual_seed(n)
    xc, xq = codes(g, min(t, 4096), d)
    xq = repeated(xq, t)
    wc, wq = codes(g, min(n, 4096), d)
    wq = repeated(wq, n)
    y = torch.full((t, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    qmm.qmm_mxfp4_gemm(packed(wq, n, d), t, n, d, xq, scales(t, d), y, n)
    want = (values(xc).double() @ values(wc).double().T).bfloat16()
    for r0 in range(0, t, xc.shape[0]):
        part = y[r0:r0 + xc.shape[0]]
        for c0 in range(0, n, wc.shape[0]):
            got = part[:, c0:c0 + wc.shape[0]]
            assert torch.equal(got, want[:got.shape[0], :got.shape[1]]), (r0, c0)


def test_quant_of_the_most_rows():
    t, d = 1 << 24, 96
    x = torch.randn(4096, d, device=DEV).bfloat16()
    q = torch.full((t, d // 2), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((t, 16), 0x55, dtype=torch.uint8, device=DEV)
    qmm.qmm_mxfp4_quant(x.repeat(t // 4096, 1), t, d, d, qmm.QMM_MX_FIT, q, s)
    qmm.qmm_mxfp4_quant(x, 4096, d, d, qmm.QMM_MX_FIT, one := torch.empty(4096, d // 2, dtype=torch.uint8, device=DEV),
                        two := torch.empty(4096, 16, dtype=torch.uint8, device=DEV))
    assert bool((q.view(-1, 4096, d // 2) == one).all()) and bool((s.view(-1, 4096, 16) == two).all())


@pytest.mark.parametrize("n_seg,rows", [(65535, 1), (65535, 3), (9000, 20)])
def test_grouped_of_the_most_segments(n_seg, rows):
    """Every other segment is empty; experts lie past 4 GiB in their stack."""
    n, d, experts, stride = 48, 64, 3, (1 << 32) + 256
    g = torch.Generator(device=DEV).manual_seed(n_seg)
    stack = torch.empty(2 * stride + 4096 * 4, dtype=torch.uint8, device=DEV)
    w = []
    for e in range(experts):
        c, q = codes(g, n, d)
        blob = packed(q, n, d)
        stack[e * stride:e * stride + blob.numel()] = blob
        w.append(values(c).double())
    full = torch.arange(n_seg, device=DEV) % 2 == 0
    lengths = torch.where(full, rows, 0)
    so = torch.zeros(n_seg + 1, dtype=torch.int32, device=DEV)
    so[1:] = lengths.cumsum(0)
    m = int(so[-1])
    se = (torch.arange(n_seg, device=DEV, dtype=torch.int32) // 2 % experts).to(torch.int32)
    xc, xq = codes(g, 500, d)
    ri = (torch.arange(m, device=DEV) * 7 % 500).to(torch.int32)
    y = guarded((m, n), float("nan"), torch.bfloat16)
    qmm.qmm_mxfp4_grouped_gemm(stack, stride, experts, n, d, xq, scales(500, d), 500, ri, se, so, n_seg, m, rows, y)
    of_row = torch.repeat_interleave(se.long(), lengths)
    each = torch.stack([values(xc).double() @ v.T for v in w])           # [expert][row of x][n]
    assert torch.equal(y, each[of_row, ri.long()].bfloat16())


#         t, E, k, d, inter: long axes, wide outputs in several rounds, the most experts and pairs
LAYERS = [(2, 3, 2, 32, 65536), (3, 2, 1, 65536, 32), (1, 2, 2, 20000, 96), (16, 1024, 16, 32, 32), (4, 80, 64, 64, 32),
          (1, 1, 1, 32, 32)]


@pytest.mark.parametrize("t,ne,k,d,inter", LAYERS)
def test_expert_layer(t, ne, k, d, inter):
    say("layer limits", t, ne, k, d, inter)
    l = Layer((t, ne, k, d, inter, "softmax", False, 1, 1, False, True, F32, 0, True), 9600 + t)
    l.check(l.run())


def test_expert_layer_past_4_gib():
    l = Layer((5, 3, 2, 96, 64, "sigmoid", False, 1, 1, False, True, F32, 0, False), 9700, pad=1 << 32)
    l.check(l.run())


def test_expert_layer_of_the_largest_activations():
    """gate and up near 2^63: h is near bf16's largest, beside it and past it."""
    l = Layer((3, 2, 2, 64, 32, "softmax", False, 1, 1, False, True, F32, 0, False), 9800)
    l.gate_up.zero_()
    c = torch.full((64, 32), 0x22, dtype=torch.uint8, device=DEV)           # every code 1
    for e in range(2):
        qmm.qmm_pack(M, 64, 64, c, torch.full((64, 2), 127, dtype=torch.uint8, device=DEV), None, l.gate_up[e])
        qmm.qmm_pack(M, 64, 32, c[:, :16].contiguous(), torch.full((64, 1), 27, dtype=torch.uint8, device=DEV), None, l.down[e])
    x = np.zeros((3, 64), np.float32)
    x[0, 0], x[1, 0], x[2, 0] = 2.0 ** 63, 1.99 * 2.0 ** 63, 2.0 ** 64
    l.x = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
    out = l.run()["out"].float()
    assert bool((out[0] == 2.0 ** 126 * 32 * 2.0 ** -100 * 2.5).all())      # both experts alike: weights 2.5 in all
    v = float(torch.tensor(1.99).bfloat16())
    assert bool(((out[1] - v * v * 2.0 ** 126 * 32 * 2.0 ** -100 * 2.5).abs() <= 2.0 ** -8 * out[1]).all())
    assert bool(torch.isinf(out[2]).all())                                  # 2^128
