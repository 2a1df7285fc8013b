"""The microscaled 4-bit calls in a row, as a layer uses them: eager, captured and replayed, on
another stream, and with profiling events (needs an MI355X)."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import bf16_to_f64, fp8, mxfp4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_fp8_profile import bracketed  # noqa: E402
from test_gpu_moe_layer import stack  # noqa: E402
from test_gpu_mxfp4 import (DEV, M, RULES, _check_guards, _gpu, as_f64, bf16_bits, dev, guarded, say,  # noqa: E402,F401
                            weights)


class Path:
    """logits -> router, quantiser, gate_up with SwiGLU, down, gather, and a dense product."""

    def __init__(self, t, ne, k, d, inter, fit, seed):
        rng = np.random.default_rng(seed)
        self.sizes = t, ne, k, d, inter
        self.fit = fit
        self.gu, self.gate_up = stack(rng, ne, 2 * inter, d)
        self.dn, self.down = stack(rng, ne, d, inter)
        self.w, self.dense = weights(rng, 96, d)
        m = t * k
        self.x, self.logits = (torch.zeros(t, n, dtype=ty, device=DEV) for n, ty in ((d, torch.bfloat16), (ne, torch.float32)))
        g = {"topk": ((t, k), torch.int32), "weights": ((t, k), torch.float32), "seg_expert": ((ne,), torch.int32),
             "seg_offsets": ((ne + 1,), torch.int32), "row_index": ((m,), torch.int32), "slot_row": ((t, k), torch.int32),
             "xq": ((t, d // 2), torch.uint8), "xs": ((t, mxfp4.scale_bytes(d)), torch.uint8),
             "hq": ((m, inter // 2), torch.uint8), "hs": ((m, mxfp4.scale_bytes(inter)), torch.uint8),
             "o": ((m, d), torch.bfloat16), "out": ((t, d), torch.bfloat16), "y": ((t, 96), torch.bfloat16)}
        self.v = {n: guarded(shape, 0, ty) for n, (shape, ty) in g.items()}
        self.ws = guarded((max(16, qmm.qmm_route_topk_workspace_bytes(t, ne)),), 0, torch.uint8)

    def inputs(self, seed):
        rng = np.random.default_rng(seed)
        t, ne, _, d, _ = self.sizes
        self.x.copy_(dev(bf16_bits(rng.normal(0, 1, (t, d)))).view(torch.bfloat16))
        self.logits.copy_(dev((rng.integers(-200, 200, (t, ne)) / 64.0).astype(np.float32)))

    def run(self, stream=None):
        t, ne, k, d, inter = self.sizes
        v, m, rule = self.v, t * k, RULES[self.fit]
        qmm.qmm_route_topk(self.logits, qmm.QMM_F32, t, ne, ne, qmm.QMM_SCORE_SOFTMAX, None, 1, 1, qmm.QMM_GROUP_MAX, k, True,
                           1.0, v["topk"], v["weights"], v["seg_expert"], v["seg_offsets"], v["row_index"], v["slot_row"],
                           self.ws, stream)
        table = (v["seg_expert"], v["seg_offsets"], ne, m, t)
        qmm.qmm_mxfp4_quant(self.x, t, d, d, rule, v["xq"], v["xs"], stream)
        qmm.qmm_mxfp4_grouped_gemm_swiglu(self.gate_up, self.gate_up.shape[1], ne, 2 * inter, d, v["xq"], v["xs"], t,
                                          v["row_index"], *table, rule, None, v["hq"], v["hs"], stream)
        qmm.qmm_mxfp4_grouped_gemm(self.down, self.down.shape[1], ne, d, inter, v["hq"], v["hs"], m, None, *table, v["o"],
                                   stream)
        qmm.qmm_moe_gather(v["o"], m, d, t, k, v["slot_row"], v["weights"], None, v["out"], stream)
        qmm.qmm_mxfp4_gemm(self.dense, t, 96, d, v["xq"], v["xs"], v["y"], 96, stream)

    def fill(self, byte):
        for x in self.v.values():
            x.view(torch.uint8).fill_(byte)

    def outputs(self):
        torch.cuda.synchronize()
        return {n: x.clone() for n, x in self.v.items()}

    def check(self):
        t, ne, k, d, inter = self.sizes
        v = {n: x.cpu() for n, x in self.outputs().items()}
        x = bf16_to_f64(self.x.cpu().view(torch.int16).numpy().view(np.uint16))
        ids, _, _ = fp8.topk(self.logits.cpu().numpy(), None, "softmax", 1, 1, False, k, True, 1.0)
        offsets, rows, slot = fp8.tables(ids, ne)
        for name, want in (("topk", ids), ("seg_offsets", offsets), ("row_index", rows), ("slot_row", slot)):
            assert np.array_equal(v[name].numpy(), want), name
        q, s = mxfp4.quant(x, self.fit)
        assert np.array_equal(v["xq"].numpy(), q) and np.array_equal(v["xs"].numpy(), s)
        xv = mxfp4.dequant(q, s)
        hq, hs = v["hq"].numpy(), v["hs"].numpy()
        hv, o = mxfp4.dequant(hq, hs), as_f64(v["o"])
        for e in range(ne):
            at = slice(offsets[e], offsets[e + 1])
            if offsets[e] == offsets[e + 1]:
                continue
            ref, rest = mxfp4.gemm(xv[rows[at]], self.gu[e])
            h, tol = mxfp4.swiglu(ref[:, :inter], ref[:, inter:], rest[:, :inter], rest[:, inter:])
            assert mxfp4.check_quantised(hq[at], hs[at], h, tol, self.fit)
            ref, rest = mxfp4.gemm(hv[at], self.dn[e])
            assert np.all(np.abs(o[at] - ref) <= mxfp4.gemm_tolerance(ref, rest))
        each = o[slot] * v["weights"].numpy().astype(np.float64)[..., None]
        assert np.all(np.abs(as_f64(v["out"]) - each.sum(1)) <= (2.0 ** -8 + k * 2.0 ** -23) * np.abs(each).sum(1) + 2.0 ** -133)
        ref, rest = mxfp4.gemm(xv, self.w)
        assert np.all(np.abs(as_f64(v["y"]) - ref) <= mxfp4.gemm_tolerance(ref, rest))


# few-row kernels; both kinds of tiles; a step's end inside a slab
SIZES = [(1, 9, 3, 96, 64), (5, 6, 2, 544, 160), (40, 4, 2, 288, 96), (150, 8, 3, 416, 224), (700, 4, 2, 1056, 512)]


@pytest.mark.parametrize("fit", [False, True])
@pytest.mark.parametrize("sizes", SIZES)
def test_the_calls_in_a_row(sizes, fit):
    say("path", sizes, fit)
    p = Path(*sizes, fit, 9100 + sizes[0])
    p.inputs(9200 + sizes[0])
    p.fill(0x55)
    p.run()
    p.check()


@pytest.mark.parametrize("sizes", [SIZES[1], SIZES[3]])
def test_graph_replays_follow_the_inputs(sizes):
    say("path graph", sizes)
    p = Path(*sizes, True, 9300)
    p.inputs(1)
    p.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for seed in range(2, 6):
        p.inputs(seed)
        p.fill(0x55)
        g.replay()
        got = p.outputs()
        p.fill(0xAA)
        p.run()
        want = p.outputs()
        for n in got:
            assert torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)), (seed, n)
    p.check()


def test_streams_of_their_own():
    """Two paths at once, each on a stream, many times over."""
    paths = [Path(*SIZES[3], True, 9400), Path(*SIZES[1], False, 9401)]
    want = []
    for n, p in enumerate(paths):
        p.inputs(n)
        p.run()
        want.append(p.outputs())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for p in paths:
            p.fill(0x55)
        torch.cuda.synchronize()
        for p, s in zip(paths, streams):
            p.run(s.cuda_stream)
        for p, w in zip(paths, want):
            for n, x in p.outputs().items():
                assert torch.equal(x.view(torch.uint8), w[n].view(torch.uint8)), n


NAMES = ["qmm_mxfp4_quant", "qmm_mxfp4_grouped_gemm_swiglu", "qmm_mxfp4_grouped_gemm", "qmm_mxfp4_gemm"]


@pytest.mark.parametrize("sizes", [SIZES[1], SIZES[4]])
@pytest.mark.parametrize("name", NAMES)
def test_events_bracket_each_call(name, sizes, monkeypatch):
    p = Path(*sizes, True, 9500)
    p.inputs(3)
    p.run()
    want = p.outputs()
    real, seen = getattr(qmm, name), []
    monkeypatch.setattr(qmm, name, lambda *a: seen.append(bracketed(lambda: real(*a))))
    p.fill(0x55)
    p.run()
    got = p.outputs()
    assert len(seen) == 1 and 0.0 < seen[0] < 100.0
    assert all(torch.equal(x.view(torch.uint8), want[n].view(torch.uint8)) for n, x in got.items())


def test_example_runs():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_moe_block.py")
    spec = importlib.util.spec_from_file_location("mxfp4_moe_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors = example.main(["--tokens", "40", "--dim", "256", "--inter", "160", "--experts", "6", "--top-k", "2"])
    # bf16 activations of up to 16 tokens: the output's rounding.  Four bits: a step of a code
    # is a third to an eighth of it, half a step at most, in x and in h
    assert errors[1] < 2.0 ** -8 and errors[16] < 2.0 ** -8 and errors[40] < 0.5
