"""Rows of routed segments: what a row gives depends on its segment's rows, not on its
place among them (needs an MI355X)."""
import numpy as np
import pytest

from oracle import fp8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_fp8 import (_check_guards, _gpu, as_f64, codes, dev, guarded, say,  # noqa: E402,F401
                          scales)


def product(rng, lengths, n, d, rows, t_x, swiglu=False):
    """One expert; the outputs, the operands."""
    m, sb = sum(lengths), fp8.blocks(n // 2)
    offs = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    w = codes(rng, 1, n, d)
    ws = scales(rng, 1, 2 * sb if swiglu else fp8.blocks(n), fp8.blocks(d)) * np.float32(0.002 if swiglu else 1.0)
    x, xs = codes(rng, t_x, d), scales(rng, t_x, fp8.blocks(d))
    y = guarded((m, n // 2 if swiglu else n), float("nan"), torch.bfloat16)
    f = qmm.qmm_fp8_grouped_gemm_swiglu if swiglu else qmm.qmm_fp8_grouped_gemm
    f(dev(w), dev(ws), 1, n, d, dev(x), dev(xs), t_x, dev(rows), dev(np.zeros(len(lengths), np.int32)), dev(offs),
      len(lengths), m, max(lengths), y)
    return y.view(torch.int16), (x, xs, w[0], ws[0])


# a last tile of 6, 16 and 17 rows after one and after two tiles of 64
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("length", [70, 80, 81, 134, 144])
def test_last_rows_of_a_segment_are_like_its_first(length, swiglu):
    say("segment", length, swiglu)
    rng = np.random.default_rng(8000 + length)
    n, d, t_x = 512, 1040, 17
    rows = (np.arange(length) % t_x).astype(np.int32)          # the same rows again and again
    short = [3, 5, 2]                                          # few rows a segment on average
    y, _ = product(rng, [length] + short, n, d, np.concatenate([rows, np.zeros(sum(short), np.int32)]), t_x, swiglu)
    y = y.cpu().numpy()[:length]
    assert np.array_equal(y, y[rows])


@pytest.mark.parametrize("length", [1, 15, 16])
def test_short_segments_have_sums_in_fp32(length):
    """Without the matrix cores' cut: 128 additions in a block in any order, two scale
    roundings, one addition a block, 16 across waves, and the rounding to bf16."""
    say("short segment", length)
    rng = np.random.default_rng(8100 + length)
    n, d, t_x = 512, 1040, 40
    lengths = [70, length, 0, length]
    rows = rng.integers(0, t_x, sum(lengths)).astype(np.int32)
    y, (x, xs, w, ws) = product(rng, lengths, n, d, rows, t_x)
    y, src = as_f64(y)[70:], rows[70:]
    ref = fp8.dequant_rows(x[src], xs[src]) @ fp8.dequant_matrix(w, ws).T
    mag = np.abs(fp8.dequant_rows(x[src], xs[src])) @ np.abs(fp8.dequant_matrix(w, ws)).T
    rest = (128 + 2 + fp8.blocks(d) + 16) * 2.0 ** -23 * mag
    assert np.all(np.abs(y - ref) <= fp8.gemm_tolerance(ref, rest))


# segments of one row take the few-row kernel, one of 4096 rows 64 x 128 tiles, and of
# 32768 rows 256 x 256 tiles
@pytest.mark.parametrize("segments_,repeat", [(4096, 1), (1, 1), (1, 8)])
def test_activation_over_its_whole_range(segments_, repeat):
    """silu(g)·g for g from -110 to 110: gate and up are the rows' scales exactly.
    Off by e^-g's (1.22·|g| + 3)·2^-24 at most, a sum, a reciprocal and two products of
    a few 2^-24, and the rounding to bf16; below 2^-126 the exponential may be zero."""
    say("silu", segments_, repeat)
    g = np.linspace(-110.0, 110.0, 4096).astype(np.float32)
    m, d, nh = 4096 * repeat, 16, 16
    x, w = np.zeros((4096, d), np.uint8), np.zeros((1, 2 * nh, d), np.uint8)
    x[:, 0], w[:, :, 0] = 0x38, 0x38                           # 1.0
    offs = np.linspace(0, m, segments_ + 1).astype(np.int32)
    h = guarded((m, nh), float("nan"), torch.bfloat16)
    qmm.qmm_fp8_grouped_gemm_swiglu(dev(w), dev(np.ones((1, 2, 1), np.float32)), 1, 2 * nh, d, dev(x), dev(g[:, None]), 4096,
                                    dev((np.arange(m) % 4096).astype(np.int32)), dev(np.zeros(segments_, np.int32)),
                                    dev(offs), segments_, m, m // segments_, h)
    h = as_f64(h.view(torch.int16))
    v = np.tile(g.astype(np.float64), repeat)[:, None]
    ref = fp8.silu(v) * v
    tol = np.abs(ref) * (2.0 ** -8 + (1.3 * np.abs(v) + 8) * 2.0 ** -23) + 2.0 ** -125 * v * v + 2.0 ** -133
    assert np.all(np.abs(h - ref) <= tol)
