"""Pins of oracle/mxfp4.py against values worked out by hand (CPU only)."""
import numpy as np

from oracle import bf16_to_f64, mxfp4


def test_rounding_to_codes():
    v = np.array([0.0, 0.25, 0.2501, 0.75, 1.25, 1.2501, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 6.0, 7.9])
    assert mxfp4.round_code(v).tolist() == [0, 0, 1, 2, 2, 3, 4, 4, 5, 6, 6, 7, 7, 7]


def test_exponents():
    """1 is 4·2^-2: E = 125.  6 fits E = 127, 6.01 needs 128; floor keeps 7.9 at 127 (saturating)."""
    m = np.array([1.0, 6.0, 6.01, 7.9, 8.0, 0.0, 2.0 ** -127, 2.0 ** 127, np.inf, np.nan])
    assert mxfp4.exponent(m, False).tolist() == [125, 127, 127, 127, 128, 0, 0, 252, 255, 255]
    assert mxfp4.exponent(m, True).tolist() == [125, 127, 128, 128, 128, 0, 0, 252, 255, 255]


def test_quant_of_a_row():
    x = np.zeros((1, 64))
    x[0, :6] = [6.0, -3.0, 0.5, -0.25, 7.0, 1.0]     # 7 saturates under floor
    q, s = mxfp4.quant(x, False)
    assert s.shape == (1, 16) and s[0, :2].tolist() == [127, 0] and not s[0, 2:].any()
    assert q[0, :3].tolist() == [0xD7, 0x81, 0x27]   # codes 7, 5|8; 1, 0|8; 7, 2
    q, s = mxfp4.quant(x, True)
    assert s[0, 0] == 128
    assert mxfp4.dequant(q, s)[0, :6].tolist() == [6.0, -3.0, 0.0, 0.0, 8.0, 1.0]   # 0.25 of 2 is a tie to 0


def test_quantised_rows_are_near():
    """fit: every value within half a step of its binade, a sixth of the block's largest at most."""
    rng = np.random.default_rng(0)
    x = rng.normal(0, 1, (20, 96))
    for fit in (False, True):
        q, s = mxfp4.quant(x, fit)
        v = mxfp4.dequant(q, s)
        if fit:
            m = np.repeat(np.abs(x).reshape(20, 3, 32).max(2), 32, 1)
            assert np.all(np.abs(v - x) <= m / 3 + 1e-12)
        assert mxfp4.check_quantised(q, s, x, np.zeros_like(x), fit)
        moved = s.copy()
        moved[0, 0] += 1
        assert not mxfp4.check_quantised(q, moved, x, np.zeros_like(x), fit)
        wrong = q.copy()
        wrong[3, 7] ^= 1
        assert not mxfp4.check_quantised(wrong, s, x, np.zeros_like(x), fit)


def test_not_finite_blocks():
    x = np.ones((2, 64))
    x[0, 3], x[1, 40] = np.inf, np.nan
    q, s = mxfp4.quant(x, False)
    assert s[:, :2].tolist() == [[255, 125], [125, 255]]
    assert not q[0, :16].any() and not q[1, 16:].any()
    assert np.isnan(mxfp4.dequant(q, s)[0, :32]).all() and np.all(mxfp4.dequant(q, s)[0, 32:] == 1.0)


def test_gemm_of_codes():
    x = np.array([[1.0, -6.0] + [0.0] * 30])
    w = np.array([[0.5, 2.0] + [0.0] * 30, [3.0, 0.5] + [0.0] * 30])
    y, rest = mxfp4.gemm(x, w)
    assert y.tolist() == [[-11.5, 0.0]] and np.all(rest > 0)
    assert np.isclose(mxfp4.silu(bf16_to_f64(np.array([0x3F80], np.uint16)))[0], 0.7310585786)
