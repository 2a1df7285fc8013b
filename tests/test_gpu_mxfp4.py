"""GPU parity of the microscaled 4-bit path against the fp64 definitions in oracle/mxfp4.py
(needs an MI355X).

Codes and exponents of the quantiser must be equal; computed numbers lie within tolerances
derived from the roundings that their definitions and kernels make.  Outputs start as a
sentinel and sit between guard bands.
"""
import sys

import numpy as np
import pytest

from oracle import bf16_to_f64, mxfp4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402

DEV = "cuda"
M = qmm.QMM_MXFP4_G32
RULES = {False: qmm.QMM_MX_FLOOR, True: qmm.QMM_MX_FIT}


def say(*a):
    print("[gpu-case]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qmm.load()
    yield
    torch.cuda.synchronize()


_guarded = []


def guarded(shape, fill, dtype, lead=256):
    """A tensor of `shape` inside a larger one whose bands hold 0x5A bytes."""
    size = torch.empty(0, dtype=dtype).element_size()
    n = int(np.prod(shape))
    base = torch.empty(lead // size + n + 4096 // size, dtype=dtype, device=DEV)
    base.view(torch.uint8).fill_(0x5A)
    body = base[lead // size:lead // size + n]
    body.fill_(fill)
    _guarded.append((base, lead, n * size))
    return body.view(*shape)


@pytest.fixture(autouse=True)
def _check_guards():
    _guarded.clear()
    yield
    torch.cuda.synchronize()
    for base, lead, n in _guarded:
        raw = base.view(torch.uint8).cpu().numpy()
        assert np.all(raw[:lead] == 0x5A) and np.all(raw[lead + n:] == 0x5A), "bytes changed outside a buffer"
    _guarded.clear()


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(DEV)


def bf16_bits(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def as_f64(t):
    return bf16_to_f64(t.view(torch.int16).cpu().numpy().view(np.uint16))


def weights(rng, n, d, lo=118, hi=126):
    """Canonical codes and exponents, and the packed blob."""
    codes = rng.integers(0, 256, (n, d // 2)).astype(np.uint8)
    e8m0 = rng.integers(lo, hi + 1, (n, d // 32)).astype(np.uint8)
    packed = torch.empty(qmm.qmm_packed_bytes(M, n, d), dtype=torch.uint8, device=DEV)
    qmm.qmm_pack(M, n, d, dev(codes), dev(e8m0), None, packed)
    return mxfp4.dequant(codes, e8m0), packed


def rows(rng, t, d, lo=119, hi=128):
    """Random codes and exponents of activation rows."""
    q = rng.integers(0, 256, (t, d // 2)).astype(np.uint8)
    s = np.zeros((t, mxfp4.scale_bytes(d)), np.uint8)
    s[:, :d // 32] = rng.integers(lo, hi + 1, (t, d // 32))
    return q, s


# ---------------------------------------------------------------- quantiser

def run_quant(bits, d, fit):
    t, ldx = bits.shape
    q = guarded((t, d // 2), 0x55, torch.uint8)
    s = guarded((t, mxfp4.scale_bytes(d)), 0x55, torch.uint8)
    qmm.qmm_mxfp4_quant(dev(bits), t, d, ldx, RULES[fit], q, s)
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("fit", [False, True])
@pytest.mark.parametrize("t,d,pad", [(1, 32, 0), (1, 512, 0), (3, 96, 8), (7, 2080, 24), (33, 5120, 0), (130, 544, 40)])
def test_quant_is_exact(t, d, pad, fit):
    say("quant", t, d, fit)
    rng = np.random.default_rng(1000 + t + d)
    v = rng.normal(0, 1, (t, d + pad)) * np.exp(rng.normal(0, 3, (t, d + pad)))
    v[0, :16] = 0.0
    v[-1, :32] = 0.0                                      # a block of zeros
    bits = bf16_bits(v)
    q, s = run_quant(bits, d, fit)
    wq, ws = mxfp4.quant(bf16_to_f64(bits)[:, :d], fit)
    assert np.array_equal(s, ws)
    assert np.array_equal(q, wq)


@pytest.mark.parametrize("fit", [False, True])
def test_quant_of_every_finite_bf16(fit):
    """Every finite pattern with every maximum's mantissa: as the largest of its block, and,
    with a larger one, at every distance where codes change; subnormals among them."""
    every = np.arange(1 << 16, dtype=np.uint16)
    every = every[(every & 0x7F80) != 0x7F80]
    alone = np.zeros((every.size, 32), np.uint16)
    alone[:, 0] = every
    rng = np.random.default_rng(3)
    near = np.abs(rng.integers(-4 * 128, 1, (every.size, 31)))
    alone[:, 1:] = np.maximum((every & 0x7FFF).astype(np.int64)[:, None] - near, 0) | (rng.integers(0, 2, near.shape) << 15)
    bits = alone.reshape(-1, 512)
    q, s = run_quant(bits, 512, fit)
    wq, ws = mxfp4.quant(bf16_to_f64(bits), fit)
    assert np.array_equal(s, ws)
    assert np.array_equal(q, wq)


@pytest.mark.parametrize("fit", [False, True])
def test_quant_infinities_and_nan_stay_in_their_block(fit):
    x = np.ones((3, 96), np.float32)
    x[0, 5], x[1, 40], x[2, 95] = np.inf, np.nan, -np.inf
    bits = bf16_bits(x)
    q, s = run_quant(bits, 96, fit)
    wq, ws = mxfp4.quant(bf16_to_f64(bits), fit)
    assert np.array_equal(s, ws) and np.array_equal(q, wq)
    assert s[0, 0] == s[1, 1] == s[2, 2] == 255


# ---------------------------------------------------------------- dense product

DENSE = [(1, 1, 32), (1, 512, 256), (1, 1000, 5120), (2, 130, 160), (5, 64, 128), (15, 257, 2080), (16, 48, 1024),
         (17, 1000, 608), (32, 300, 4096), (33, 77, 5152), (64, 256, 640), (65, 129, 1056), (128, 128, 128),
         (130, 513, 2080), (257, 260, 416), (300, 1000, 608), (511, 640, 288), (777, 1029, 1184)]


def dense(t, n, d, seed, ldy=None, lead=256):
    rng = np.random.default_rng(seed)
    w, packed = weights(rng, n, d)
    q, s = rows(rng, t, d)
    ldy = ldy or n
    y = guarded((t, ldy), float("nan"), torch.bfloat16, lead)
    qmm.qmm_mxfp4_gemm(packed, t, n, d, dev(q), dev(s), y, ldy)
    ref, rest = mxfp4.gemm(mxfp4.dequant(q, s), w)
    return as_f64(y), ref, mxfp4.gemm_tolerance(ref, rest)


@pytest.mark.parametrize("t,n,d", DENSE)
def test_gemm(t, n, d):
    say("gemm", t, n, d)
    y, ref, tol = dense(t, n, d, 7 + t + n + d)
    assert np.all(np.abs(y - ref) <= tol), np.max(np.abs(y - ref) / tol)


@pytest.mark.parametrize("t,n,d,ldy,lead", [(3, 70, 96, 75, 256), (40, 33, 544, 64, 258), (300, 129, 288, 131, 2)])
def test_gemm_row_stride(t, n, d, ldy, lead):
    y, ref, tol = dense(t, n, d, 50 + t, ldy, lead)
    assert np.all(np.abs(y[:, :n] - ref) <= tol)
    assert np.all(np.isnan(y[:, n:]))


@pytest.mark.parametrize("t", [1, 40, 300])
def test_gemm_of_whole_numbers_is_exact(t):
    """Codes of whole values with one exponent: every sum is a whole number below 2^24, so
    nothing but the rounding to bf16 may be off, whatever the order."""
    n, d = 200, 1120
    rng = np.random.default_rng(t)
    wc = rng.choice([0, 2, 4, 5, 6, 7, 10, 12, 15], (n, d)).astype(np.uint8)
    xc = rng.choice([0, 2, 4, 5, 6, 7, 10, 12, 15], (t, d)).astype(np.uint8)
    we = np.full((n, d // 32), 127, np.uint8)
    s = np.zeros((t, mxfp4.scale_bytes(d)), np.uint8)
    s[:, :d // 32] = 127
    packed = torch.empty(qmm.qmm_packed_bytes(M, n, d), dtype=torch.uint8, device=DEV)
    wq, xq = mxfp4.pack_codes(wc), mxfp4.pack_codes(xc)
    qmm.qmm_pack(M, n, d, dev(wq), dev(we), None, packed)
    y = guarded((t, n), float("nan"), torch.bfloat16)
    qmm.qmm_mxfp4_gemm(packed, t, n, d, dev(xq), dev(s), y, n)
    want = mxfp4.dequant(xq, s) @ mxfp4.dequant(wq, we).T
    assert np.array_equal(as_f64(y), bf16_to_f64(bf16_bits(want)))


@pytest.mark.parametrize("t", [2, 300])
def test_gemm_exponents_far_apart(t):
    """Exponents over their range; products stay inside fp32's."""
    n, d = 130, 1056
    rng = np.random.default_rng(90 + t)
    w, packed = weights(rng, n, d, 60, 190)
    q, s = rows(rng, t, d, 70, 180)
    y = guarded((t, n), 0.0, torch.bfloat16)
    qmm.qmm_mxfp4_gemm(packed, t, n, d, dev(q), dev(s), y, n)
    ref, rest = mxfp4.gemm(mxfp4.dequant(q, s), w)
    assert np.all(np.abs(as_f64(y) - ref) <= mxfp4.gemm_tolerance(ref, rest))


@pytest.mark.parametrize("t", [1, 20, 50, 300])
def test_gemm_nan_blocks_make_their_row_nan(t):
    """An exponent of 255 in the first and in the last block, d ending inside a step; the
    codes of a NaN block are zeros, as the quantiser writes them."""
    n, d = 70, 544 + 32
    rng = np.random.default_rng(91)
    w, packed = weights(rng, n, d)
    q, s = rows(rng, t, d)
    for row, b in ((0, 0), (t - 1, d // 32 - 1)):
        s[row, b] = 255
        q[row, 16 * b:16 * b + 16] = 0
    y = guarded((t, n), 0.0, torch.bfloat16)
    qmm.qmm_mxfp4_gemm(packed, t, n, d, dev(q), dev(s), y, n)
    y = as_f64(y)
    assert np.isnan(y[0]).all() and np.isnan(y[t - 1]).all() and np.isfinite(y[1:t - 1]).all()


# ---------------------------------------------------------------- grouped products

def stack(rng, experts, n, d):
    size = qmm.qmm_packed_bytes(M, n, d)
    blob = torch.empty(experts * size, dtype=torch.uint8, device=DEV)
    ws = []
    for e in range(experts):
        w, p = weights(rng, n, d)
        blob[e * size:(e + 1) * size] = p
        ws.append(w)
    return ws, blob, size


GROUPED = [  # n, d, lengths of the segments
    (64, 96, [1, 0, 2]), (128, 544, [0, 0, 1, 1, 3]), (192, 2080, [5, 17, 0, 1]), (128, 288, [64, 1, 33, 0, 16]),
    (576, 1056, [70, 0, 130, 257, 3]), (1024, 512, [300, 20, 500, 1]), (64, 32, [1] * 300)]


def tables(rng, lengths, t_x, experts):
    m = sum(lengths)
    offs = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return (rng.integers(0, experts, len(lengths)).astype(np.int32), offs, rng.integers(0, t_x, m).astype(np.int32), m)


@pytest.mark.parametrize("indexed", [True, False])
@pytest.mark.parametrize("n,d,lengths", GROUPED)
def test_grouped(n, d, lengths, indexed):
    say("grouped", n, d, lengths[:6], indexed)
    rng = np.random.default_rng(n + d)
    experts = 3
    ws, blob, size = stack(rng, experts, n, d)
    m = sum(lengths)
    t_x = 11 if indexed else m
    se, so, ri, m = tables(rng, lengths, t_x, experts)
    if not indexed:
        ri = np.arange(m, dtype=np.int32)
    q, s = rows(rng, t_x, d)
    y = guarded((m, n), float("nan"), torch.bfloat16)
    qmm.qmm_mxfp4_grouped_gemm(blob, size, experts, n, d, dev(q), dev(s), t_x, dev(ri) if indexed else None, dev(se),
                               dev(so), len(lengths), m, max(lengths), y)
    got, x = as_f64(y), mxfp4.dequant(q, s)
    for i, e in enumerate(se):
        at = slice(so[i], so[i + 1])
        ref, rest = mxfp4.gemm(x[ri[at]], ws[e])
        assert np.all(np.abs(got[at] - ref) <= mxfp4.gemm_tolerance(ref, rest)), i


@pytest.mark.parametrize("fit", [None, False, True])
@pytest.mark.parametrize("n,d,lengths", GROUPED)
def test_grouped_swiglu(n, d, lengths, fit):
    say("swiglu", n, d, lengths[:6], fit)
    rng = np.random.default_rng(n + d + 1)
    experts, t_x, i = 3, 13, n // 2
    ws, blob, size = stack(rng, experts, n, d)
    se, so, ri, m = tables(rng, lengths, t_x, experts)
    q, s = rows(rng, t_x, d, 117, 122)
    table = (dev(ri), dev(se), dev(so), len(lengths), m, max(lengths))
    x = mxfp4.dequant(q, s)
    if fit is None:
        h = guarded((m, i), float("nan"), torch.bfloat16)
        qmm.qmm_mxfp4_grouped_gemm_swiglu(blob, size, experts, n, d, dev(q), dev(s), t_x, *table, 0, h, None, None)
        got = as_f64(h)
    else:
        hq = guarded((m, i // 2), 0x55, torch.uint8)
        hs = guarded((m, mxfp4.scale_bytes(i)), 0x55, torch.uint8)
        qmm.qmm_mxfp4_grouped_gemm_swiglu(blob, size, experts, n, d, dev(q), dev(s), t_x, *table, RULES[fit], None, hq, hs)
        codes, exps = hq.cpu().numpy(), hs.cpu().numpy()
    for k, e in enumerate(se):
        at = slice(so[k], so[k + 1])
        if so[k] == so[k + 1]:
            continue
        y, rest = mxfp4.gemm(x[ri[at]], ws[e])
        want, tol = mxfp4.swiglu(y[:, :i], y[:, i:], rest[:, :i], rest[:, i:])
        if fit is None:
            assert np.all(np.abs(got[at] - want) <= 2.0 ** -8 * (np.abs(want) + tol) + tol)
        else:
            assert mxfp4.check_quantised(codes[at], exps[at], want, tol, fit)


@pytest.mark.parametrize("length", [2, 20, 200])
def test_grouped_bad_tables(length):
    """Experts and rows out of range give NaN, rows that no segment covers stay as they were,
    offsets past m_total are held back."""
    n, d, experts, t_x = 128, 288, 2, 5
    rng = np.random.default_rng(8)
    ws, blob, size = stack(rng, experts, n, d)
    q, s = rows(rng, t_x, d)
    lengths = [length] * 4
    m = sum(lengths) + 3                                     # three rows behind the last segment
    se = np.array([0, 2, -1, 1], np.int32)
    so = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    ri = rng.integers(0, t_x, m).astype(np.int32)
    ri[0], ri[1] = -1, t_x
    table = (dev(ri), dev(se), dev(so), 4, m, length)
    y = guarded((m, n), 0.5, torch.bfloat16)
    qmm.qmm_mxfp4_grouped_gemm(blob, size, experts, n, d, dev(q), dev(s), t_x, *table, y)
    got = as_f64(y)
    nan = np.zeros(m, bool)
    nan[[0, 1]] = True
    nan[length:3 * length] = True
    assert np.isnan(got[nan]).all() and np.isfinite(got[~nan]).all() and np.all(got[-3:] == 0.5)
    hq = guarded((m, n // 4), 0x55, torch.uint8)
    hs = guarded((m, mxfp4.scale_bytes(n // 2)), 0x55, torch.uint8)
    qmm.qmm_mxfp4_grouped_gemm_swiglu(blob, size, experts, n, d, dev(q), dev(s), t_x, *table, 1, None, hq, hs)
    c, e = hq.cpu().numpy(), hs.cpu().numpy()
    assert np.all(e[nan][:, :n // 64] == 255) and not c[nan].any()
    assert np.all(c[-3:] == 0x55) and np.all(e[-3:] == 0x55)
    assert not np.any(e[:-3][:, :n // 64][~nan[:-3]] == 255)
    so2 = so.copy()
    so2[-1] = 1 << 30
    y2 = guarded((m, n), 0.5, torch.bfloat16)
    qmm.qmm_mxfp4_grouped_gemm(blob, size, experts, n, d, dev(q), dev(s), t_x, dev(ri), dev(se), dev(so2), 4, m, length + 3, y2)
    assert np.isfinite(as_f64(y2)[3 * length:]).all() and not np.any(as_f64(y2)[-3:] == 0.5)
