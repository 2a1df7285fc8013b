"""Pins of the fp64 definitions in oracle/fp8.py: the e4m3 code table and its
rounding, a hand-worked quantisation and product, and the router's choice,
weights and tables on tiny inputs."""
import numpy as np

from oracle import fp8


def test_e4m3_table():
    v = fp8.e4m3_to_f64(np.arange(256))
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[7] == 7 * 2.0 ** -9 and v[8] == 2.0 ** -6
    assert v[0x38] == 1.0 and v[0x39] == 1.125 and v[0x7E] == 448.0 and np.isnan(v[0x7F]) and np.isnan(v[0xFF])
    assert np.array_equal(-v[:127], v[128:255])
    assert np.all(np.diff(v[:127]) > 0)


def test_e4m3_rounding():
    code = lambda x: int(fp8.f64_to_e4m3(x))  # noqa: E731
    for c in range(127):                                  # every value is its own code
        assert code(fp8.e4m3_to_f64(c)) == c and code(-fp8.e4m3_to_f64(c)) == c | 0x80
    assert code(1.0625) == 0x38 and code(1.1875) == 0x3A  # midway: the even code
    assert code(2.0 ** -10) == 0 and code(1.5 * 2.0 ** -9) == 2
    assert code(450.0) == 0x7E and code(np.nan) == 0x7F


def test_quant_by_hand():
    x = np.zeros((1, 130), np.float32)
    x[0, 0], x[0, 1], x[0, 129] = 896.0, -1.0, 0.0
    q, s = fp8.quant(x)
    assert s[0, 0] == 2.0 and s[0, 1] == np.float32(2.0 ** -96) / np.float32(448)
    v = fp8.dequant_rows(q, s)
    assert v[0, 0] == 896.0 and v[0, 1] == -1.0 and np.all(v[0, 2:] == 0.0)


def test_gemm_by_hand():
    x = np.full((1, 144), 0x38, np.uint8)                  # ones
    w = np.full((130, 144), 0x40, np.uint8)                # twos
    xs = np.array([[1.0, 10.0]], np.float32)
    ws = np.array([[1.0, 2.0], [3.0, 0.5]], np.float32)
    y, rest = fp8.gemm(x, xs, w, ws)
    assert y[0, 0] == 128 * 2 * 1.0 + 16 * 2 * 10.0 * 2.0 and y[0, 129] == 128 * 2 * 3.0 + 16 * 2 * 10.0 * 0.5
    group = lambda c: 16 * 2 * c[0] + 2 * 2 * c[1]  # noqa: E731  (16 groups of 8 products of 2, then 2 groups)
    a = group((1.0, 20.0)) * 8
    assert a == y[0, 0]
    assert np.isclose(rest[0, 0], (128 + 2 + 2 + 16) * 2.0 ** -23 * a + 7 * 2.0 ** -13 * a / 8)


def test_topk_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w, _ = fp8.topk(l, None, "softmax", 1, 1, False, 2, False, 1.0)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 0.25]])
    ids, w, _ = fp8.topk(l, None, "softmax", 1, 1, False, 3, True, 2.0)
    assert ids.tolist() == [[2, 1, 0]]                     # equal logits: the lower expert
    assert np.allclose(w, 2.0 * np.array([[4, 2, 1]]) / 7)
    # groups {0,1} and {2,3}: largest 4 against 2, sums of two 5 against 3
    ids, _, _ = fp8.topk(l, None, "softmax", 2, 1, False, 3, False, 1.0)
    assert ids.tolist() == [[2, 3, -1]]
    # sigmoid: the bias changes the choice and not the weight
    z = np.zeros((1, 4))
    ids, w, _ = fp8.topk(z, np.array([0.0, 0.0, 0.0, 1.0]), "sigmoid", 2, 1, True, 1, False, 1.0)
    assert ids.tolist() == [[3]] and w[0, 0] == 0.5
    # masked: never chosen, and a row with nothing left
    l = np.array([[-np.inf, 0.0, -np.inf, 0.0], [-np.inf] * 4])
    for score in ("softmax", "sigmoid"):
        ids, w, _ = fp8.topk(l, None, score, 1, 1, False, 3, True, 1.0)
        assert ids.tolist() == [[1, 3, -1], [-1, -1, -1]]
        assert np.allclose(w, [[0.5, 0.5, 0], [0, 0, 0]])


def test_tables_by_hand():
    offsets, rows, slot = fp8.tables(np.array([[2, 0], [2, -1], [0, 1]], np.int32), 3)
    assert offsets.tolist() == [0, 2, 3, 5]
    assert rows.tolist() == [0, 2, 2, 0, 1, -1]
    assert slot.tolist() == [[3, 0], [4, -1], [1, 2]]


def test_norm_by_hand():
    v, h = fp8.norm_residual(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), np.array([[2.0, 1.0]]),
                             np.array([[1.0, 1.0]]), 0.5, np.array([0.0, 0.0]), 1.0, 0.0)
    k = 1.0 / np.sqrt(12.5)
    assert np.allclose(v, [[0.5 + 2.0 * 3.0 * k * 2.0, 0.5 + 4.0 * k * 3.0]])
    assert np.allclose((h * h).mean(), 1.0)


def test_gemm_tolerance_holds_a_half_ulp():
    y = np.array([1.0, -300.0])
    tol = fp8.gemm_tolerance(y, np.zeros(2))
    assert np.all(tol >= 2.0 ** -8 * np.abs(y)) and np.all(tol < 2.0 ** -7 * np.abs(y))
