"""GPU parity of the block-scaled e4m3 path, the top-k router, the gather and
the norms against the fp64 definitions in oracle/fp8.py (needs an MI355X).

Codes and tables must be equal; computed numbers lie within tolerances derived
from the roundings that their definitions and kernels make (oracle/fp8.py).
Outputs start as a sentinel and sit between guard bands.
"""
import sys

import numpy as np
import pytest

from oracle import bf16_to_f64, fp8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402

DEV = "cuda"
BF, F32 = qmm.QMM_BF16, qmm.QMM_F32


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
    return bf16_to_f64(t.cpu().numpy().view(np.uint16))


def codes(rng, *shape):
    """Random finite e4m3 codes, zeros and both signs among them."""
    c = rng.integers(0, 127, shape).astype(np.uint8)
    return c | (rng.integers(0, 2, shape).astype(np.uint8) << 7)


def scales(rng, *shape):
    return np.exp(rng.normal(-5.0, 1.0, shape)).astype(np.float32)


# ---------------------------------------------------------------- quantiser

@pytest.mark.parametrize("t,d,pad", [(1, 16, 0), (1, 128, 0), (3, 144, 8), (7, 2064, 24), (33, 5120, 0), (130, 272, 40)])
def test_quant_is_exact(t, d, pad):
    say("quant", t, d)
    rng = np.random.default_rng(1000 + t + d)
    v = rng.normal(0, 1, (t, d + pad)) * np.exp(rng.normal(0, 3, (t, d + pad)))
    v[0, :16] = 0.0                                       # a block of zeros where d is 16
    v[-1, :min(d, 128)] *= 2.0 ** -120                    # a block under the floor
    bits = bf16_bits(v)
    x = bf16_to_f64(bits)[:, :d]
    q = guarded((t, d), 0x55, torch.uint8)
    s = guarded((t, fp8.blocks(d)), float("nan"), torch.float32)
    qmm.qmm_fp8_quant(dev(bits), t, d, d + pad, q, s)
    wq, ws = fp8.quant(x)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)


def test_quant_range_and_ties():
    """The largest and smallest bf16, maxima of every exponent, and values midway between codes."""
    rows = [np.concatenate([[2.0 ** e * (1 + m / 128)], 2.0 ** e * np.arange(127) / 127.0])
            for e in range(-90, 127, 7) for m in (0, 1, 127)]
    rows.append(np.concatenate([[448.0], np.arange(1, 128) * 0.5]))
    bits = bf16_bits(np.array(rows))
    x = bf16_to_f64(bits)
    t, d = x.shape
    q, s = guarded((t, d), 0x55, torch.uint8), guarded((t, 1), 0.0, torch.float32)
    qmm.qmm_fp8_quant(dev(bits), t, d, d, q, s)
    wq, ws = fp8.quant(x)
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


def test_quant_infinities_and_nan_stay_in_their_block():
    x = np.ones((3, 384), np.float32)
    x[0, 5], x[1, 200], x[2, 383] = np.inf, np.nan, -np.inf
    q, s = guarded((3, 384), 0, torch.uint8), guarded((3, 3), 0.0, torch.float32)
    qmm.qmm_fp8_quant(dev(bf16_bits(x)), 3, 384, 384, q, s)
    v = q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 1)
    v = v.cpu().numpy()
    hit = np.zeros((3, 3), bool)
    hit[0, 0] = hit[1, 1] = hit[2, 2] = True
    hit = np.repeat(hit, 128, 1)
    assert np.all(np.isnan(v[hit])) and np.all(v[~hit] == 1.0)


# ---------------------------------------------------------------- dense product

DENSE = [(1, 1, 16), (1, 512, 256), (1, 1000, 5120), (2, 130, 144), (5, 64, 128), (15, 257, 2064), (16, 48, 1024),
         (17, 1000, 592), (32, 300, 4096), (33, 77, 5136), (64, 256, 640), (65, 129, 1040), (128, 128, 128),
         (130, 513, 2064), (257, 260, 400), (300, 1000, 592), (511, 640, 272), (777, 1029, 1168)]


def dense(t, n, d, seed, ldy=None, lead=256):
    rng = np.random.default_rng(seed)
    x, w = codes(rng, t, d), codes(rng, n, d)
    xs, ws = scales(rng, t, fp8.blocks(d)), scales(rng, fp8.blocks(n), fp8.blocks(d))
    ldy = ldy or n
    y = guarded((t, ldy), float("nan"), torch.bfloat16, lead)
    qmm.qmm_fp8_gemm(dev(w), dev(ws), t, n, d, dev(x), dev(xs), y, ldy)
    ref, rest = fp8.gemm(x, xs, w, ws)
    return as_f64(y.view(torch.int16)), ref, fp8.gemm_tolerance(ref, rest)


@pytest.mark.parametrize("t,n,d", DENSE)
def test_gemm_parity(t, n, d):
    say("fp8 gemm", t, n, d)
    y, ref, tol = dense(t, n, d, 2000 + t + n + d)
    worst = np.max(np.abs(y - ref) / tol)
    say("worst / tolerance", worst)
    assert worst <= 1.0


@pytest.mark.parametrize("t,n,d,ldy,lead", [(3, 30, 128, 37, 256), (70, 130, 256, 144, 256), (300, 250, 384, 251, 258),
                                            (300, 256, 384, 256, 258)])
def test_gemm_strides(t, n, d, ldy, lead):
    y, ref, tol = dense(t, n, d, 2500 + t, ldy, lead)
    assert np.all(np.abs(y[:, :n] - ref) <= tol) and np.all(np.isnan(y[:, n:]))


@pytest.mark.parametrize("t", [1, 20, 64, 200, 600])
def test_gemm_integers_are_exact(t):
    """Small whole numbers with scales of powers of two: every sum is exact, so every bit is known."""
    rng = np.random.default_rng(2600 + t)
    n, d = 300, 1040
    x = fp8.f64_to_e4m3(rng.integers(-2, 3, (t, d)).astype(float))
    w = fp8.f64_to_e4m3(rng.integers(-2, 3, (n, d)).astype(float))
    xs = np.exp2(rng.integers(-1, 2, (t, 9))).astype(np.float32)
    ws = np.exp2(rng.integers(-1, 2, (3, 9))).astype(np.float32)
    y = guarded((t, n), float("nan"), torch.bfloat16)
    qmm.qmm_fp8_gemm(dev(w), dev(ws), t, n, d, dev(x), dev(xs), y, n)
    ref, _ = fp8.gemm(x, xs, w, ws)
    want = torch.from_numpy(ref.astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy()
    assert np.array_equal(y.view(torch.int16).cpu().numpy(), want)


@pytest.mark.parametrize("t", [2, 40, 300])
def test_gemm_nan_stays_in_its_row_and_column(t):
    rng = np.random.default_rng(2700 + t)
    n, d = 200, 400
    x, w = codes(rng, t, d), codes(rng, n, d)
    xs, ws = scales(rng, t, 4), scales(rng, 2, 4)
    x[1, 399], w[77, 0], xs[0, 2] = 0x7F, 0xFF, np.inf
    y = guarded((t, n), 0.0, torch.bfloat16)
    qmm.qmm_fp8_gemm(dev(w), dev(ws), t, n, d, dev(x), dev(xs), y, n)
    y = as_f64(y.view(torch.int16))
    bad = ~np.isfinite(y)
    assert bad[1].all() and bad[:, 77].all() and bad[0].all()
    bad[1], bad[0], bad[:, 77] = False, False, False
    assert not bad.any()


@pytest.mark.parametrize("t", [1, 33, 600])
def test_gemm_repeats_bitwise(t):
    rng = np.random.default_rng(2800 + t)
    n, d = 700, 1040
    a = [dev(v) for v in (codes(rng, n, d), scales(rng, 6, 9), codes(rng, t, d), scales(rng, t, 9))]
    outs = []
    for _ in range(3):
        y = guarded((t, n), float("nan"), torch.bfloat16)
        qmm.qmm_fp8_gemm(a[0], a[1], t, n, d, a[2], a[3], y, n)
        outs.append(y.view(torch.int16).cpu().numpy())
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


# ---------------------------------------------------------------- grouped product

def segments(rng, lengths, ne, t_x):
    offs = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    experts = rng.integers(0, ne, len(lengths)).astype(np.int32)
    rows = rng.integers(0, t_x, offs[-1]).astype(np.int32)
    return experts, offs, rows


GROUPED = [([1, 0, 1, 1], 48, 128), ([5, 3, 0, 16, 1], 130, 272), ([17, 2, 33], 257, 144), ([64, 0, 65, 7], 96, 1040),
           ([130, 1, 300, 40], 260, 528), ([0, 0, 1], 16, 16), ([257, 511], 640, 272)]


@pytest.mark.parametrize("index", [True, False])
@pytest.mark.parametrize("bound", ["exact", "tokens", "one"])
@pytest.mark.parametrize("lengths,n,d", GROUPED)
def test_grouped_parity(lengths, n, d, bound, index):
    say("fp8 grouped", lengths, n, d, bound, index)
    rng = np.random.default_rng(3000 + n + d)
    ne, m = 3, sum(lengths)
    t_x = 37 if index else m
    experts, offs, rows = segments(rng, lengths, ne, t_x)
    w, ws = codes(rng, ne, n, d), scales(rng, ne, fp8.blocks(n), fp8.blocks(d))
    x, xs = codes(rng, t_x, d), scales(rng, t_x, fp8.blocks(d))
    y = guarded((m, n), float("nan"), torch.bfloat16)
    most = {"exact": max(lengths), "tokens": m, "one": 1}[bound]      # the bound never limits what is computed
    qmm.qmm_fp8_grouped_gemm(dev(w), dev(ws), ne, n, d, dev(x), dev(xs), t_x, dev(rows) if index else None,
                             dev(experts), dev(offs), len(lengths), m, most, y)
    y = as_f64(y.view(torch.int16))
    for i, e in enumerate(experts):
        at = slice(offs[i], offs[i + 1])
        src = rows[at] if index else np.arange(offs[i], offs[i + 1])
        ref, rest = fp8.gemm(x[src], xs[src], w[e], ws[e])
        assert np.all(np.abs(y[at] - ref) <= fp8.gemm_tolerance(ref, rest)), i


@pytest.mark.parametrize("bound", ["exact", "tokens"])
@pytest.mark.parametrize("lengths,nh,d", [([1, 1, 0, 2], 32, 128), ([20, 3], 200, 272), ([70, 130, 1, 33], 136, 400),
                                          ([300, 5], 257, 144)])
def test_grouped_swiglu_parity(lengths, nh, d, bound):
    say("fp8 swiglu", lengths, nh, d)
    rng = np.random.default_rng(3500 + nh + d)
    ne, m, t_x, nb, sb = 3, sum(lengths), 29, fp8.blocks(d), fp8.blocks(nh)
    experts, offs, rows = segments(rng, lengths, ne, t_x)
    w, ws = codes(rng, ne, 2 * nh, d), scales(rng, ne, 2 * sb, nb) * np.float32(0.002)
    x, xs = codes(rng, t_x, d), scales(rng, t_x, nb) * np.float32(0.1)
    h = guarded((m, nh), float("nan"), torch.bfloat16)
    qmm.qmm_fp8_grouped_gemm_swiglu(dev(w), dev(ws), ne, 2 * nh, d, dev(x), dev(xs), t_x, dev(rows), dev(experts),
                                    dev(offs), len(lengths), m, max(lengths) if bound == "exact" else m, h)
    h = as_f64(h.view(torch.int16))
    for i, e in enumerate(experts):
        at = slice(offs[i], offs[i + 1])
        if not lengths[i]:
            continue
        g, gr = fp8.gemm(x[rows[at]], xs[rows[at]], w[e, :nh], ws[e, :sb])
        u, ur = fp8.gemm(x[rows[at]], xs[rows[at]], w[e, nh:], ws[e, sb:])
        assert np.abs(g).max() < 40
        ref, tol = fp8.swiglu_tolerance(g, u, gr, ur)
        assert np.all(np.abs(h[at] - ref) <= tol), i


@pytest.mark.parametrize("length", [4, 90, 300])
def test_grouped_bad_experts_and_rows(length):
    rng = np.random.default_rng(3600 + length)
    ne, n, d, t_x = 2, 130, 144, 11
    lengths = [length, length, length]
    m = sum(lengths)
    experts, offs, rows = segments(rng, lengths, ne, t_x)
    experts[:] = [0, 2, -1]
    rows[1], rows[2] = t_x, -1
    offs[-1] = m + 50                                     # past the end: clamped
    w, ws = codes(rng, ne, n, d), scales(rng, ne, 2, 2)
    x, xs = codes(rng, t_x, d), scales(rng, t_x, 2)
    y = guarded((m, n), 1.0, torch.bfloat16)
    qmm.qmm_fp8_grouped_gemm(dev(w), dev(ws), ne, n, d, dev(x), dev(xs), t_x, dev(rows), dev(experts), dev(offs), 3, m,
                             m, y)
    y = as_f64(y.view(torch.int16))
    good = np.ones(m, bool)
    good[[1, 2]] = False
    good[length:] = False
    assert np.isnan(y[~good]).all()
    src = rows[good]
    ref, rest = fp8.gemm(x[src], xs[src], w[0], ws[0])
    assert np.all(np.abs(y[good] - ref) <= fp8.gemm_tolerance(ref, rest))


def test_grouped_uncovered_rows_are_left_alone():
    rng = np.random.default_rng(3700)
    n, d, m = 48, 128, 20
    offs, experts = np.array([3, 3, 9], np.int32), np.array([0, 0], np.int32)
    w, ws, x, xs = codes(rng, 1, n, d), scales(rng, 1, 1, 1), codes(rng, m, d), scales(rng, m, 1)
    for most in (1, m):
        y = guarded((m, n), 7.0, torch.bfloat16)
        qmm.qmm_fp8_grouped_gemm(dev(w), dev(ws), 1, n, d, dev(x), dev(xs), m, None, dev(experts), dev(offs), 2, m, most, y)
        y = as_f64(y.view(torch.int16))
        assert np.all(y[:3] == 7.0) and np.all(y[9:] == 7.0) and not np.any(y[3:9] == 7.0)


# ---------------------------------------------------------------- router

def route(l, dtype, ld, score, bias, groups, keep, top2, k, renorm, scale):
    t, ne = l.shape
    full = np.full((t, ld), 50.0, np.float32)
    full[:, :ne] = l
    full = torch.from_numpy(full).to(DEV)
    if dtype == BF:
        full = full.to(torch.bfloat16)
    out = {"topk": guarded((t, k), -7, torch.int32), "weights": guarded((t, k), float("nan"), torch.float32),
           "seg_expert": guarded((ne,), -7, torch.int32), "seg_offsets": guarded((ne + 1,), -7, torch.int32),
           "row_index": guarded((t * k,), -7, torch.int32), "slot_row": guarded((t, k), -7, torch.int32)}
    need = qmm.qmm_route_topk_workspace_bytes(t, ne)
    ws = guarded((need,), 0xEE, torch.uint8) if need else None
    qmm.qmm_route_topk(full, dtype, t, ne, ld, qmm.QMM_SCORE_SIGMOID if score == "sigmoid" else qmm.QMM_SCORE_SOFTMAX,
                       None if bias is None else torch.from_numpy(bias).to(DEV), groups, keep,
                       qmm.QMM_GROUP_TOP2 if top2 else qmm.QMM_GROUP_MAX, k, renorm, scale, *out.values(), ws)
    torch.cuda.synchronize()
    return {n: v.cpu().numpy() for n, v in out.items()}


# (tokens, experts, k, score, bias, groups, keep, top2, renorm, type, ld - experts)
ROUTES = [(1, 1, 1, "softmax", False, 1, 1, False, True, F32, 0), (1, 256, 8, "sigmoid", True, 8, 4, True, True, F32, 0),
          (5, 60, 4, "softmax", False, 1, 1, False, False, F32, 3), (128, 64, 6, "softmax", False, 8, 3, False, True, BF, 0),
          (129, 160, 6, "softmax", False, 8, 3, False, True, F32, 8), (300, 256, 8, "sigmoid", True, 8, 4, True, True, BF, 1),
          (33, 384, 8, "sigmoid", True, 12, 5, False, True, F32, 0), (200, 896, 16, "sigmoid", True, 1, 1, False, True, F32, 0),
          (3, 1024, 64, "sigmoid", False, 64, 20, True, False, F32, 0), (77, 72, 5, "softmax", True, 8, 2, True, True, F32, 0),
          (40, 9, 9, "sigmoid", False, 3, 2, True, True, F32, 0), (2500, 40, 3, "softmax", False, 40, 7, True, False, F32, 0),
          (5000, 16, 2, "sigmoid", True, 2, 1, True, True, BF, 0), (64, 512, 8, "softmax", False, 4, 1, False, True, F32, 0)]


@pytest.mark.parametrize("case", ROUTES)
def test_route_parity(case):
    t, ne, k, score, with_bias, groups, keep, top2, renorm, dtype, pad = case
    say("route", case)
    rng = np.random.default_rng(4000 + t + ne)
    # logits on a grid: no two of a row closer than 2^-6 unless they are equal (exact ties, the lower expert first)
    l = rng.integers(-200, 200, (t, ne)) / 64.0
    bias = (rng.integers(-8, 9, ne) / 32.0).astype(np.float32) if with_bias else None
    l[rng.random((t, ne)) < 0.1] = -np.inf
    l[t // 2] = -np.inf if t > 4 else l[t // 2]            # a token with nothing left
    if dtype == BF:
        l = bf16_to_f64(bf16_bits(l))
    ids, w, gap = fp8.topk(l, bias, score, groups, keep, top2, k, renorm, 2.5)
    got = route(l, dtype, ne + pad, score, bias, groups, keep, top2, k, renorm, 2.5)
    # fp32 scores carry a few 2^-24 of error, sums and biases a few more; rows whose
    # choice hangs on less than that are only checked for their weights
    clear = gap > 64 * 2.0 ** -24
    assert clear.mean() > 0.9
    assert np.array_equal(got["topk"][clear], ids[clear])
    tol = (np.abs(w) + 1e-30) * (ne + 64) * 2.0 ** -23
    assert np.all(np.abs(got["weights"] - w)[clear] <= tol[clear])
    offsets, rows, slot = fp8.tables(got["topk"], ne) if t * k * ne < 4e6 else tables_fast(got["topk"], ne)
    assert np.array_equal(got["seg_expert"], np.arange(ne)) and np.array_equal(got["seg_offsets"], offsets)
    assert np.array_equal(got["row_index"], rows) and np.array_equal(got["slot_row"], slot)


def tables_fast(ids, ne):
    flat = np.where(ids.reshape(-1) < 0, ne, ids.reshape(-1))
    order = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=ne + 1)[:ne])]).astype(np.int32)
    slot = np.empty(flat.size, np.int32)
    slot[order] = np.arange(flat.size)
    k = ids.shape[1]
    return offsets, np.where(flat[order] < ne, order // k, -1).astype(np.int32), \
        np.where(ids < 0, -1, slot.reshape(ids.shape)).astype(np.int32)


@pytest.mark.parametrize("t", [1, 129, 20000])
def test_route_large_tables(t):
    rng = np.random.default_rng(4500 + t)
    ne, k = 256, 8
    l = rng.normal(0, 1, (t, ne)).astype(np.float32)
    got = route(l, F32, ne, "softmax", None, 8, 4, False, k, True, 1.0)
    offsets, rows, slot = tables_fast(got["topk"], ne)
    assert np.array_equal(got["seg_offsets"], offsets) and np.array_equal(got["row_index"], rows)
    assert np.array_equal(got["slot_row"], slot)
    best = l.reshape(t, 8, 32).max(-1)
    kept = np.argsort(-best, 1, kind="stable")[:, :4]
    c = np.full((t, 8, 32), -np.inf, np.float32)
    np.put_along_axis(c, kept[:, :, None], np.take_along_axis(l.reshape(t, 8, 32), kept[:, :, None], 1), 1)
    assert np.array_equal(got["topk"], np.argsort(-c.reshape(t, ne), 1, kind="stable")[:, :k])


def test_route_values_at_the_edges():
    """Lowest finite logits, infinities, signed zeros and NaN."""
    low, inf, nan = -3.4028235e38, np.inf, np.nan
    l = np.array([[low, low, low, low], [0.0, -0.0, -1.0, 0.0], [inf, 1.0, 2.0, -inf], [nan, 1.0, -inf, 0.0],
                  [low, -inf, 3.0, low]], np.float32)
    got = route(l, F32, 4, "sigmoid", None, 1, 1, False, 3, True, 1.0)
    assert got["topk"].tolist() == [[0, 1, 2], [0, 1, 3], [0, 2, 1], [1, 3, -1], [2, 0, 3]]
    assert np.all(got["weights"][0] == 0.0)               # their sum is 0
    assert got["weights"][4].tolist() == [1.0, 0.0, 0.0] and got["weights"][3, 2] == 0.0
    got = route(l, F32, 4, "softmax", None, 1, 1, False, 3, False, 1.0)
    assert got["topk"].tolist() == [[0, 1, 2], [0, 1, 3], [0, 2, 1], [1, 3, -1], [2, 0, 3]]
    assert np.all(got["weights"][0] == 0.25) and np.isnan(got["weights"][2]).any()
    assert np.isnan(got["weights"][3, :2]).all() and got["weights"][3, 2] == 0.0
    assert got["weights"][4].tolist() == [1.0, 0.0, 0.0]


def test_route_no_tokens():
    so, se = guarded((9,), -7, torch.int32), guarded((8,), -7, torch.int32)
    qmm.qmm_route_topk(None, F32, 0, 8, 8, 0, None, 1, 1, 0, 2, True, 1.0, None, None, se, so, None, None, None)
    assert so.tolist() == [0] * 9 and se.tolist() == list(range(8))


# ---------------------------------------------------------------- gather

@pytest.mark.parametrize("t,k,d,shared", [(1, 1, 8, False), (4, 8, 3584, True), (33, 3, 2056, False), (9, 17, 264, True)])
def test_gather_parity(t, k, d, shared):
    rng = np.random.default_rng(5000 + t + d)
    m = t * k + 3
    ob, sb = bf16_bits(rng.normal(0, 1, (m, d))), bf16_bits(rng.normal(0, 1, (t, d)))
    slot = rng.permutation(m)[:t * k].reshape(t, k).astype(np.int32)
    slot[rng.random((t, k)) < 0.2] = -1
    slot[t - 1] = -1                                      # a token that no expert took
    w = rng.random((t, k)).astype(np.float32)
    out = guarded((t, d), float("nan"), torch.bfloat16)
    qmm.qmm_moe_gather(dev(ob), m, d, t, k, dev(slot), dev(w), dev(sb) if shared else None, out)
    o = bf16_to_f64(ob)
    terms = np.where(slot[..., None] >= 0, w[..., None].astype(float) * o[np.maximum(slot, 0)], 0.0)
    add = bf16_to_f64(sb) if shared else 0.0
    ref, mag = terms.sum(1) + add, np.abs(terms).sum(1) + np.abs(add)
    got = as_f64(out.view(torch.int16))
    rest = (k + 1) * 2.0 ** -24 * mag
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + rest) + rest + 2.0 ** -133)


def test_gather_bad_slot():
    o = torch.ones(3, 16, dtype=torch.bfloat16, device=DEV)
    slot = torch.tensor([[0, 3], [1, 2]], dtype=torch.int32, device=DEV)
    out = guarded((2, 16), 0.0, torch.bfloat16)
    qmm.qmm_moe_gather(o, 3, 16, 2, 2, slot, torch.ones(2, 2, device=DEV), None, out)
    assert torch.isnan(out[0]).all() and (out[1] == 2.0).all()


# ---------------------------------------------------------------- norms

def norm_tolerance(h_ref, v_ref, dv, d):
    """h from a v that is off by dv: the mean square moves by at most 2·|v|·dv a
    term; fp32 sums of d squares, a square root, a division and three products."""
    ms = (v_ref ** 2).mean(1, keepdims=True)
    dms = 2.0 * (np.abs(v_ref) * dv).mean(1, keepdims=True) + (dv ** 2).mean(1, keepdims=True)
    rel = 0.5 * dms / np.maximum(ms, 1e-300) + (d // 8 + 24) * 2.0 ** -24
    scale = np.abs(h_ref) / np.maximum(np.abs(v_ref), 1e-300)
    return scale * dv + np.abs(h_ref) * (rel + 8 * 2.0 ** -24)


# (tokens, width, residual type, post weights, gate rows (0: none), block output, offset, h, codes, in place)
NORMS = [(1, 8, BF, True, 1, True, 0.0, True, True, False), (1, 5120, BF, True, 1, True, 0.0, True, True, False),
         (7, 136, F32, True, 3, True, 1.0, True, True, True), (5, 520, BF, False, 0, True, 0.0, True, False, True),
         (3, 2064, F32, True, 100, True, 1.0, False, True, False), (4, 4104, BF, False, 2, True, 0.0, True, True, False),
         (2, 8200, BF, True, 0, True, 0.0, True, True, True), (2, 16392, F32, True, 1, True, 0.0, True, True, False),
         (1, 65536, BF, True, 1, True, 0.0, True, True, False), (6, 256, BF, False, 0, False, 0.0, True, True, False),
         (3, 264, BF, True, 1, True, 0.0, False, False, False)]


@pytest.mark.parametrize("case", NORMS)
def test_norm_parity(case):
    t, d, rt, post, gate_rows, with_o, offset, with_h, with_q, in_place = case
    say("norm", case)
    rng = np.random.default_rng(6000 + t + d)
    pad = 8
    b = lambda *s: bf16_bits(rng.normal(0, 1, s))  # noqa: E731
    ob, w1b, w2b = b(t, d + pad), b(d), b(d)
    rows = -(-t // gate_rows) if gate_rows else 0
    gb = b(rows, d + 2 * pad) if rows else None
    r = rng.normal(0, 2, (t, d + pad)).astype(np.float32)
    if rt == BF:
        r = bf16_to_f64(bf16_bits(r)).astype(np.float32)
    if t > 2:
        r[1] = 0.0                                        # a row of zeros: eps alone under the root
        ob[1] = 0
    tt = torch.bfloat16 if rt == BF else torch.float32
    rd = guarded((t, d + pad), 0.0, tt)
    rd.copy_(torch.from_numpy(r))
    out = rd if in_place else guarded((t, d + pad), 5.0, tt)
    h = guarded((t, d + pad), float("nan"), torch.bfloat16) if with_h else None
    q = guarded((t, d), 0x55, torch.uint8) if with_q else None
    s = guarded((t, fp8.blocks(d)), float("nan"), torch.float32) if with_q else None
    qmm.qmm_norm_residual(t, d, dev(ob) if with_o else None, d + pad, dev(w1b) if post else None,
                          dev(gb) if rows else None, d + 2 * pad, max(1, gate_rows), rd, rt, d + pad, 0.75, out, d + pad,
                          dev(w2b) if with_h or with_q else None, offset, 1e-6, h, d + pad, q, s)
    f = lambda x: bf16_to_f64(x)  # noqa: E731
    gate = f(gb)[:, :d][np.arange(t) // gate_rows] if rows else None
    o = f(ob)[:, :d] if with_o else None
    v, want = fp8.norm_residual(o, f(w1b) if post else None, gate, r[:, :d], 0.75, f(w2b), offset, 1e-6)
    # v: the sum of squares ((d/8 + 24) roundings at most), root, division, products, gate, residual
    u = v - 0.75 * r[:, :d].astype(float)
    dv = np.abs(u) * ((d // 8 + 24) * 2.0 ** -24 + 8 * 2.0 ** -24) + (np.abs(v) + np.abs(u)) * 2.0 ** -23
    got = out.float().cpu().numpy().astype(float)
    half = 2.0 ** -8 if rt == BF else 2.0 ** -24
    assert np.all(np.abs(got[:, :d] - v) <= half * (np.abs(v) + dv) + dv + 1e-40)
    if not in_place:
        assert np.all(got[:, d:] == 5.0)
    dh = norm_tolerance(want, v, dv, d) + 1e-40
    if with_h:
        gh = as_f64(h.view(torch.int16))
        assert np.all(np.abs(gh[:, :d] - want) <= 2.0 ** -8 * (np.abs(want) + dh) + dh) and np.all(np.isnan(gh[:, d:]))
    if with_q:
        # each code is the nearest to some value within dh of h; the scale that of a maximum within its block's dh
        codes_, sc = q.cpu().numpy(), s.cpu().numpy().astype(float)
        val = fp8.e4m3_to_f64(codes_)
        step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(val), 2.0 ** -6))) - 3), 2.0 ** -9)
        full = np.repeat(sc, 128, 1)[:, :d]
        assert np.all(np.abs(val * full - want) <= 0.5 * step * full * (1 + 2.0 ** -20) + dh * (1 + 2.0 ** -3))
        for blk in range(fp8.blocks(d)):
            at = slice(128 * blk, min(d, 128 * blk + 128))
            m = np.maximum(np.abs(want[:, at]).max(1), fp8.FLOOR)
            assert np.all(np.abs(sc[:, blk] * 448.0 - m) <= dh[:, at].max(1) + m * 2.0 ** -22)


def test_norm_codes_are_those_of_the_quantiser():
    """With weights and rows that make h a bf16 number exactly, the fused codes equal the quantiser's."""
    t, d = 5, 640
    rng = np.random.default_rng(6500)
    sign = rng.integers(0, 2, (t, d)) * 2.0 - 1.0
    w = bf16_bits(rng.normal(0, 1, d))
    r = torch.from_numpy(sign.astype(np.float32)).to(DEV)       # mean square 1, eps 0: h = ±w
    h, q = guarded((t, d), 0.0, torch.bfloat16), guarded((t, d), 0, torch.uint8)
    s = guarded((t, 5), 0.0, torch.float32)
    qmm.qmm_norm_residual(t, d, None, d, None, None, 0, 1, r, F32, d, 1.0, None, d, dev(w), 0.0, 0.0, h, d, q, s)
    wq, ws = fp8.quant(sign * bf16_to_f64(w))
    assert np.array_equal(as_f64(h.view(torch.int16)), sign * bf16_to_f64(w))
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


# ---------------------------------------------------------------- streams and graphs

def layer(t, ne, k, d, inter, seed):
    """Every call of one routed block on buffers made once; returns (inputs, outputs, run)."""
    rng = np.random.default_rng(seed)
    m = t * k
    b = {"o": torch.empty(t, d, dtype=torch.bfloat16, device=DEV), "r": torch.empty(t, d, dtype=torch.bfloat16, device=DEV),
         "l": torch.empty(t, ne, device=DEV)}
    w2 = dev(bf16_bits(1 + 0.1 * rng.normal(0, 1, d)))
    gu, gus = dev(codes(rng, ne, 2 * inter, d)), dev(scales(rng, ne, 2 * fp8.blocks(inter), fp8.blocks(d)) * np.float32(1e-3))
    dn, dns = dev(codes(rng, ne, d, inter)), dev(scales(rng, ne, fp8.blocks(d), fp8.blocks(inter)) * np.float32(1e-2))
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    bf, u8, i4 = torch.bfloat16, torch.uint8, torch.int32
    v = {"v": e(t, d, dt=bf), "h": e(t, d, dt=bf), "q": e(t, d, dt=u8), "s": e(t, fp8.blocks(d)), "topk": e(t, k, dt=i4),
         "weights": e(t, k), "seg_expert": e(ne, dt=i4), "seg_offsets": e(ne + 1, dt=i4), "row_index": e(m, dt=i4),
         "slot_row": e(t, k, dt=i4), "a": e(m, inter, dt=bf), "aq": e(m, inter, dt=u8), "as": e(m, fp8.blocks(inter)),
         "y": e(m, d, dt=bf), "out": e(t, d, dt=bf), "dense": e(t, 2 * inter, dt=bf)}
    ws = e(max(1, qmm.qmm_route_topk_workspace_bytes(t, ne)), dt=u8)

    def run(stream=None):
        tab = (v["seg_expert"], v["seg_offsets"], ne, m, t)
        qmm.qmm_norm_residual(t, d, b["o"], d, w2, None, 0, 1, b["r"], BF, d, 1.0, v["v"], d, w2, 0.0, 1e-6, v["h"], d,
                              v["q"], v["s"], stream=stream)
        qmm.qmm_route_topk(b["l"], F32, t, ne, ne, 1, None, 1, 1, 0, k, True, 1.0, v["topk"], v["weights"],
                           v["seg_expert"], v["seg_offsets"], v["row_index"], v["slot_row"], ws, stream=stream)
        qmm.qmm_fp8_grouped_gemm_swiglu(gu, gus, ne, 2 * inter, d, v["q"], v["s"], t, v["row_index"], *tab, v["a"],
                                        stream=stream)
        qmm.qmm_fp8_quant(v["a"], m, inter, inter, v["aq"], v["as"], stream=stream)
        qmm.qmm_fp8_grouped_gemm(dn, dns, ne, d, inter, v["aq"], v["as"], m, None, *tab, v["y"], stream=stream)
        qmm.qmm_moe_gather(v["y"], m, d, t, k, v["slot_row"], v["weights"], v["h"], v["out"], stream=stream)
        qmm.qmm_fp8_gemm(gu, gus, t, 2 * inter, d, v["q"], v["s"], v["dense"], 2 * inter, stream=stream)

    def fill(s):
        g = np.random.default_rng(s)
        b["o"].copy_(torch.from_numpy(g.normal(0, 1, (t, d)).astype(np.float32)))
        b["r"].copy_(torch.from_numpy(g.normal(0, 1, (t, d)).astype(np.float32)))
        b["l"].copy_(torch.from_numpy(g.normal(0, 1, (t, ne)).astype(np.float32)))

    def reset():
        for x in v.values():
            x.fill_(0 if not x.is_floating_point() else float("nan"))

    return v, run, fill, reset


@pytest.mark.parametrize("t", [3, 200])
def test_graph_replay_matches_eager(t):
    say("fp8 graph", t)
    v, run, fill, reset = layer(t, 12, 4, 256, 144, 7000 + t)
    fill(1)
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for s in (2, 3, 4):
        fill(s)
        reset()
        run()
        torch.cuda.synchronize()
        want = {n: x.clone() for n, x in v.items()}
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for n, x in v.items():
            assert torch.equal(x.view(torch.uint8), want[n].view(torch.uint8)), n


def test_calls_on_another_stream():
    v, run, fill, reset = layer(150, 12, 4, 256, 144, 7100)
    fill(5)
    reset()
    run()
    torch.cuda.synchronize()
    want = {n: x.clone() for n, x in v.items()}
    reset()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    run(stream=side)
    side.synchronize()
    for n, x in v.items():
        assert torch.equal(x.view(torch.uint8), want[n].view(torch.uint8)), n


def test_profile_events_bracket_every_call():
    import ctypes
    hip = ctypes.CDLL("libamdhip64.so")
    ev = [ctypes.c_void_p(), ctypes.c_void_p()]
    for e in ev:
        assert hip.hipEventCreate(ctypes.byref(e)) == 0
    v, run, fill, reset = layer(200, 12, 4, 256, 144, 7200)
    fill(6)
    l, ws = torch.randn(200, 12, device=DEV), torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    qmm.qmm_profile_next(ev[0].value, ev[1].value)
    qmm.qmm_route_topk(l, F32, 200, 12, 12, 1, None, 1, 1, 0, 4, True, 1.0, v["topk"], v["weights"], v["seg_expert"],
                       v["seg_offsets"], v["row_index"], v["slot_row"], ws)
    torch.cuda.synchronize()
    ms = ctypes.c_float(-1.0)
    assert hip.hipEventElapsedTime(ctypes.byref(ms), ev[0], ev[1]) == 0 and 0.0 < ms.value < 100.0
    for e in ev:
        hip.hipEventDestroy(e)
