"""GPU parity of the block-scaled e4m3 products where they run on the large tiles,
with every height of a part tile, and with more segments than one look at the
table holds (needs an MI355X).  Tolerances: oracle/fp8.py."""
import numpy as np
import pytest

from oracle import fp8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_fp8 import (_check_guards, _gpu, as_f64, codes, dense, dev, guarded, say,  # noqa: E402,F401
                          scales, segments)


# 2048 rows are whole tiles; the rest is a part tile of up to a quarter, half, three quarters, or more
@pytest.mark.parametrize("rest", [1, 64, 65, 128, 129, 192, 193, 255])
def test_part_tiles_of_a_dense_product(rest):
    say("large tile", rest)
    y, ref, tol = dense(2048 + rest, 6001, 336, 4000 + rest)
    assert np.max(np.abs(y - ref) / tol) <= 1.0


def test_large_product_of_integers_is_exact():
    rng = np.random.default_rng(4100)
    t, n, d = 2100, 6000, 400
    x = fp8.f64_to_e4m3(rng.integers(-2, 3, (t, d)).astype(float))
    w = fp8.f64_to_e4m3(rng.integers(-2, 3, (n, d)).astype(float))
    xs = np.exp2(rng.integers(-1, 2, (t, 4))).astype(np.float32)
    ws = np.exp2(rng.integers(-1, 2, (47, 4))).astype(np.float32)
    y = guarded((t, n), float("nan"), torch.bfloat16)
    qmm.qmm_fp8_gemm(dev(w), dev(ws), t, n, d, dev(x), dev(xs), y, n)
    ref = fp8.dequant_rows(x, xs) @ fp8.dequant_matrix(w, ws).T
    want = torch.from_numpy(ref.astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy()
    assert np.array_equal(y.view(torch.int16).cpu().numpy(), want)


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 300, 320, 385, 449, 513] + [60] * 10
MANY = [(7 * i) % 11 for i in range(300)]
MANY_LONG = [40 + (37 * i) % 101 for i in range(300)]


@pytest.mark.parametrize("lengths,n,d", [(LENGTHS, 1030, 400), (MANY, 72, 144), (MANY_LONG, 40, 80)])
def test_grouped_tiles(lengths, n, d):
    say("grouped tiles", len(lengths), n, d)
    rng = np.random.default_rng(4200 + n)
    ne, m, t_x = 5, sum(lengths), 211
    experts, offs, rows = segments(rng, lengths, ne, t_x)
    rows[::50] = t_x                                          # rows without a source
    w, ws = codes(rng, ne, n, d), scales(rng, ne, fp8.blocks(n), fp8.blocks(d))
    x, xs = codes(rng, t_x, d), scales(rng, t_x, fp8.blocks(d))
    y = guarded((m, n), 0.0, torch.bfloat16)
    qmm.qmm_fp8_grouped_gemm(dev(w), dev(ws), ne, n, d, dev(x), dev(xs), t_x, dev(rows), dev(experts), dev(offs),
                             len(lengths), m, max(lengths), y)
    y = as_f64(y.view(torch.int16))
    bad = rows == t_x
    assert np.isnan(y[bad]).all()
    rows[bad] = 0
    for i, e in enumerate(experts):
        at = slice(offs[i], offs[i + 1])
        ref, rest = fp8.gemm(x[rows[at]], xs[rows[at]], w[e], ws[e])
        ok = np.abs(y[at] - ref) <= fp8.gemm_tolerance(ref, rest)
        assert np.all(ok | bad[at][:, None]), (i, lengths[i])


@pytest.mark.parametrize("nh,d", [(520, 400)])
def test_grouped_swiglu_tiles(nh, d):
    say("swiglu tiles", nh, d)
    rng = np.random.default_rng(4300)
    lengths = LENGTHS
    ne, m, t_x, nb, sb = 3, sum(lengths), 101, fp8.blocks(d), fp8.blocks(nh)
    experts, offs, rows = segments(rng, lengths, ne, t_x)
    experts[7] = ne                                           # no such expert
    w, ws = codes(rng, ne, 2 * nh, d), scales(rng, ne, 2 * sb, nb) * np.float32(0.002)
    x, xs = codes(rng, t_x, d), scales(rng, t_x, nb) * np.float32(0.1)
    h = guarded((m, nh), 0.0, torch.bfloat16)
    qmm.qmm_fp8_grouped_gemm_swiglu(dev(w), dev(ws), ne, 2 * nh, d, dev(x), dev(xs), t_x, dev(rows), dev(experts),
                                    dev(offs), len(lengths), m, max(lengths), h)
    h = as_f64(h.view(torch.int16))
    for i, e in enumerate(experts):
        at = slice(offs[i], offs[i + 1])
        if e == ne:
            assert np.isnan(h[at]).all()
            continue
        g, rg = fp8.gemm(x[rows[at]], xs[rows[at]], w[e][:nh], ws[e][:sb])
        u, ru = fp8.gemm(x[rows[at]], xs[rows[at]], w[e][nh:], ws[e][sb:])
        want, tol = fp8.swiglu_tolerance(g, u, rg, ru)
        assert np.all(np.abs(h[at] - want) <= tol), (i, lengths[i])
