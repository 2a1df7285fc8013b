"""GPU parity of the few-token mixture-of-experts layer against the fp64 definitions of the
router (oracle/fp8.py) and of the experts (oracle/moe.py) (needs an MI355X)."""
import numpy as np
import pytest

from oracle import bf16_to_f64, fp8, moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_mxfp4 import (DEV, M, _check_guards, _gpu, as_f64, bf16_bits, dev, guarded, say,  # noqa: E402,F401
                            weights)

BF, F32 = qmm.QMM_BF16, qmm.QMM_F32


def stack(rng, ne, n, d, pad=0):
    """Dequantised matrices and their packed stack, rows of `pad` bytes more than needed."""
    size = qmm.qmm_packed_bytes(M, n, d) + pad
    out, w = torch.full((ne, size), 0xA5, dtype=torch.uint8, device=DEV), []
    for e in range(ne):
        m, blob = weights(rng, n, d)
        out[e, :blob.numel()] = blob
        w.append(m)
    return w, out


class Layer:
    def __init__(self, case, seed, pad=0):
        (self.t, self.ne, self.k, self.d, self.inter, self.score, bias, self.groups, self.keep, self.top2, self.renorm,
         self.dtype, self.ld_pad, shared) = case
        rng = np.random.default_rng(seed)
        self.gu, self.gate_up = stack(rng, self.ne, 2 * self.inter, self.d, pad)
        self.dn, self.down = stack(rng, self.ne, self.d, self.inter, pad)
        self.x = bf16_bits(rng.normal(0, 1, (self.t, self.d)))
        # on a grid: no two logits of a token closer than 2^-6 unless they are equal
        self.logits = rng.integers(-200, 200, (self.t, self.ne)) / 64.0
        if self.dtype == BF:
            self.logits = bf16_to_f64(bf16_bits(self.logits))
        self.bias = (rng.integers(-8, 9, self.ne) / 32.0).astype(np.float32) if bias else None
        self.shared = bf16_bits(rng.normal(0, 1, (self.t, self.d))) if shared else None
        self.scale = 2.5

    def buffers(self):
        return {"topk": guarded((self.t, self.k), -7, torch.int32),
                "weights": guarded((self.t, self.k), float("nan"), torch.float32),
                "out": guarded((self.t, self.d), float("nan"), torch.bfloat16, 264),
                "ws": guarded((qmm.qmm_moe_layer_workspace_bytes(self.t, self.k, self.inter),), 0xFF, torch.uint8)}

    def inputs(self):
        ld = self.ne + self.ld_pad
        l = np.full((self.t, ld), 50.0, np.float32)
        l[:, :self.ne] = self.logits
        l = torch.from_numpy(l).to(DEV)
        return {"x": dev(self.x).view(torch.bfloat16), "logits": l.to(torch.bfloat16) if self.dtype == BF else l, "ld": ld,
                "bias": None if self.bias is None else dev(self.bias),
                "shared": None if self.shared is None else dev(self.shared).view(torch.bfloat16)}

    def call(self, i, o, stream=None):
        qmm.qmm_moe_layer(M, self.gate_up, self.gate_up.shape[1], self.down, self.down.shape[1], self.ne, self.d,
                          self.inter, i["x"], self.t, i["logits"], self.dtype, i["ld"],
                          qmm.QMM_SCORE_SIGMOID if self.score == "sigmoid" else qmm.QMM_SCORE_SOFTMAX, i["bias"],
                          self.groups, self.keep, qmm.QMM_GROUP_TOP2 if self.top2 else qmm.QMM_GROUP_MAX, self.k,
                          self.renorm, self.scale, i["shared"], o["topk"], o["weights"], o["out"], o["ws"], stream)

    def run(self):
        o = self.buffers()
        self.call(self.inputs(), o)
        torch.cuda.synchronize()
        return o

    def check(self, o, clear_share=0.9):
        ids, w, gap = fp8.topk(self.logits, self.bias, self.score, self.groups, self.keep, self.top2, self.k, self.renorm,
                               self.scale)
        clear = gap > 64 * 2.0 ** -24
        assert clear.mean() >= clear_share
        got, gw = o["topk"].cpu().numpy(), o["weights"].cpu().numpy().astype(np.float64)
        assert np.array_equal(got[clear], ids[clear])
        tol = (np.abs(w) + 1e-30) * (self.ne + 64) * 2.0 ** -23
        assert np.all(np.abs(gw - w)[clear] <= tol[clear])
        shared = None if self.shared is None else bf16_to_f64(self.shared)
        want, tol = moe.layer(bf16_to_f64(self.x), self.gu, self.dn, got, gw, shared)
        off = np.abs(as_f64(o["out"]) - want)
        assert np.all(off <= tol), np.nanmax(off / tol)


#         t, E, k, d, inter, score, bias, groups, keep, top2, renorm, logits, pad, shared
CASES = [(1, 1, 1, 32, 32, "softmax", False, 1, 1, False, True, F32, 0, False),
         (1, 24, 8, 512, 256, "sigmoid", True, 8, 4, True, True, F32, 0, True),
         (2, 8, 2, 1024, 512, "softmax", False, 1, 1, False, True, F32, 0, False),
         (3, 64, 64, 96, 32, "sigmoid", False, 1, 1, False, False, BF, 3, True),
         (4, 5, 2, 128, 160, "softmax", True, 1, 1, False, True, F32, 1, True),
         (5, 6, 6, 640, 608, "softmax", False, 3, 3, True, True, BF, 0, False),
         (7, 20, 4, 2080, 1056, "softmax", False, 1, 1, False, False, BF, 4, True),
         (8, 3, 2, 544, 1120, "sigmoid", True, 1, 1, False, True, F32, 0, False),
         (9, 300, 8, 64, 32, "sigmoid", True, 12, 5, False, True, F32, 0, True),
         (12, 40, 20, 288, 96, "softmax", False, 1, 1, False, True, F32, 0, False),
         (13, 700, 5, 32, 64, "softmax", False, 7, 3, True, True, BF, 2, False),
         (16, 16, 16, 160, 96, "sigmoid", False, 4, 4, False, True, F32, 0, True),
         (16, 64, 8, 1568, 288, "softmax", False, 1, 1, False, True, BF, 0, False),
         (16, 4, 1, 4128, 32, "softmax", False, 1, 1, False, False, F32, 0, True),
         (16, 2, 2, 1600, 2208, "sigmoid", False, 2, 2, True, True, F32, 0, False)]


@pytest.mark.parametrize("case", CASES)
def test_layer(case):
    say("moe layer", case)
    l = Layer(case, 8000 + case[0] + case[1] + case[3], pad=256 * (case[0] % 3))
    l.check(l.run())


@pytest.mark.parametrize("t", [1, 4, 5, 8, 9, 16])
def test_every_token_to_one_expert(t):
    l = Layer((t, 7, 1, 672, 352, "softmax", False, 1, 1, False, True, F32, 0, True), 8100 + t)
    l.logits[:] = 0.0
    l.logits[:, 5] = 1.0
    o = l.run()
    assert np.all(o["topk"].cpu().numpy() == 5)
    l.check(o)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_tokens_with_few_experts_or_none_left(score):
    l = Layer((11, 30, 6, 352, 192, score, False, 1, 1, False, True, F32, 0, True), 8200)
    rng = np.random.default_rng(8201)
    for i in range(11):
        left = rng.choice(30, min(i, 8), replace=False)
        row = np.full(30, -np.inf)
        row[left] = l.logits[i, left]
        l.logits[i] = row
    o = l.run()
    assert np.all(o["topk"].cpu().numpy()[0] == -1)
    l.check(o)
    assert torch.equal(o["out"][0], dev(l.shared).view(torch.bfloat16)[0])


def test_nothing_chosen_at_all():
    for shared in (False, True):
        l = Layer((3, 9, 2, 96, 64, "softmax", False, 1, 1, False, True, F32, 0, shared), 8300)
        l.logits[:] = -np.inf
        o = l.run()
        assert bool((o["topk"] == -1).all()) and bool((o["weights"] == 0).all())
        want = dev(l.shared).view(torch.bfloat16) if shared else torch.zeros(3, 96, dtype=torch.bfloat16, device=DEV)
        assert torch.equal(o["out"], want)


def test_equal_logits_go_to_the_lowest_experts():
    l = Layer((6, 12, 5, 64, 32, "sigmoid", False, 1, 1, False, True, F32, 0, False), 8400)
    l.logits[:] = 0.25
    o = l.run()
    assert np.array_equal(o["topk"].cpu().numpy(), np.tile(np.arange(5), (6, 1)))
    l.check(o, 0.0)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_bad_activations_stay_in_their_token(bad):
    case = (9, 6, 3, 416, 224, "softmax", False, 1, 1, False, True, F32, 0, False)
    l = Layer(case, 8500)
    good = l.run()
    l.x[4, 77] = bf16_bits(np.array([bad]))[0]
    o = l.run()
    keep = [i for i in range(9) if i != 4]
    assert torch.equal(o["out"][keep], good["out"][keep])
    assert not bool(torch.isfinite(o["out"][4].float()).any())


def test_nan_logits():
    """Never chosen; under softmax the token's weights are NaN, and so is its output."""
    l = Layer((4, 10, 3, 96, 64, "softmax", False, 1, 1, False, True, F32, 0, False), 8600)
    l.logits[2, 4] = np.nan
    o = l.run()
    assert not bool((o["topk"][2] == 4).any())
    assert bool(torch.isnan(o["weights"][2]).all()) and bool(torch.isnan(o["out"][2].float()).all())
    keep = [0, 1, 3]
    assert bool(torch.isfinite(o["out"][keep].float()).all())
    l = Layer((4, 10, 3, 96, 64, "sigmoid", False, 1, 1, False, True, F32, 0, False), 8600)
    l.logits[2, 4] = np.nan
    l.check(l.run())


def test_shared_may_be_the_output():
    l = Layer((5, 9, 3, 224, 128, "softmax", False, 1, 1, False, True, F32, 0, True), 8700)
    want = l.run()["out"]
    i, o = l.inputs(), l.buffers()
    o["out"].copy_(i["shared"])
    i["shared"] = o["out"]
    l.call(i, o)
    assert torch.equal(o["out"], want)


def test_same_results_each_time_and_beside_another_call():
    """Two layers at once on two streams, each with its own workspace, many times over."""
    a = Layer((16, 20, 6, 800, 416, "softmax", False, 1, 1, False, True, F32, 0, True), 8800)
    b = Layer((3, 12, 4, 1248, 640, "sigmoid", True, 4, 2, True, True, BF, 0, False), 8801)
    want = [l.run() for l in (a, b)]
    a.check(want[0])
    b.check(want[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[l.buffers() for _ in range(10)] for l in (a, b)]
    ins = [l.inputs() for l in (a, b)]
    torch.cuda.synchronize()
    for r in range(10):
        for n, l in enumerate((a, b)):
            with torch.cuda.stream(streams[n]):
                l.call(ins[n], got[n][r])
    torch.cuda.synchronize()
    for n in range(2):
        for o in got[n]:
            for key in ("topk", "weights", "out"):
                assert torch.equal(o[key], want[n][key]), key


def test_graph_replays_follow_the_inputs():
    """One captured layer, replayed with the router's and the activations' values changed."""
    l = Layer((6, 14, 3, 480, 256, "softmax", False, 1, 1, False, True, F32, 0, True), 8900)
    i, o = l.inputs(), l.buffers()
    l.call(i, o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        l.call(i, o)
    rng = np.random.default_rng(8901)
    for r in range(4):
        l.logits = rng.integers(-200, 200, (l.t, l.ne)) / 64.0
        l.x = bf16_bits(rng.normal(0, 1, (l.t, l.d)))
        fresh = l.inputs()
        i["logits"].copy_(fresh["logits"])
        i["x"].copy_(fresh["x"])
        for key in ("topk", "weights", "out", "ws"):
            o[key].fill_(3)
        g.replay()
        torch.cuda.synchronize()
        want = l.run()
        for key in ("topk", "weights", "out"):
            assert torch.equal(o[key], want[key]), (r, key)
        l.check(o)


def test_agrees_with_the_calls_it_joins():
    """Router, grouped SwiGLU product, grouped product and gather with bf16 activations make
    the same choice; their outputs differ by the bf16 rounding of each expert's output."""
    case = (16, 24, 4, 1184, 544, "sigmoid", True, 6, 3, True, True, F32, 0, True)
    l = Layer(case, 9000)
    o, i = l.run(), l.inputs()
    l.check(o)
    t, k, ne, d, inter = l.t, l.k, l.ne, l.d, l.inter
    m = t * k
    topk, w = torch.empty(t, k, dtype=torch.int32, device=DEV), torch.empty(t, k, device=DEV)
    seg_e, seg_o = torch.empty(ne, dtype=torch.int32, device=DEV), torch.empty(ne + 1, dtype=torch.int32, device=DEV)
    rows, slot = torch.empty(m, dtype=torch.int32, device=DEV), torch.empty(t, k, dtype=torch.int32, device=DEV)
    qmm.qmm_route_topk(i["logits"], F32, t, ne, i["ld"], qmm.QMM_SCORE_SIGMOID, i["bias"], 6, 3, qmm.QMM_GROUP_TOP2, k, True,
                       l.scale, topk, w, seg_e, seg_o, rows, slot, None)
    assert torch.equal(topk, o["topk"]) and torch.equal(w, o["weights"])
    h = torch.empty(m, inter, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(m, d, dtype=torch.bfloat16, device=DEV)
    qmm.qmm_grouped_gemm_swiglu(M, l.gate_up, l.gate_up.shape[1], ne, 2 * inter, d, i["x"], t, rows, seg_e, seg_o, ne, m, t, h)
    qmm.qmm_grouped_gemm(M, l.down, l.down.shape[1], ne, d, inter, h, m, None, seg_e, seg_o, ne, m, t, y)
    out = torch.empty(t, d, dtype=torch.bfloat16, device=DEV)
    qmm.qmm_moe_gather(y, m, d, t, k, slot, w, i["shared"], out)
    got = [bf16_to_f64(bf16_bits(v.float().cpu().numpy())) for v in (out, o["out"])]
    want, tol = moe.layer(bf16_to_f64(l.x), l.gu, l.dn, topk.cpu().numpy(), w.cpu().numpy().astype(np.float64),
                          bf16_to_f64(l.shared))
    each = np.abs(y.float().cpu().numpy().astype(np.float64))[slot.cpu().numpy()]       # [t][k][d]
    extra = 2.0 ** -8 * 1.02 * (np.abs(w.cpu().numpy())[..., None] * each).sum(1)
    assert np.all(np.abs(got[0] - got[1]) <= 2 * tol + extra)


def test_events_bracket_both_launches():
    from test_gpu_fp8_profile import bracketed
    l = Layer((16, 24, 6, 1568, 800, "softmax", False, 1, 1, False, True, F32, 0, True), 9050)
    i, o = l.inputs(), l.buffers()
    l.call(i, o)
    want = o["out"].clone()
    o["out"].fill_(0)
    assert 0.0 < bracketed(lambda: l.call(i, o)) < 100.0
    assert torch.equal(o["out"], want)
