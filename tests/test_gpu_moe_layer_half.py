"""GPU parity of the expert layer in half of its workspace (needs an MI355X)."""
import functools
from unittest import mock

import numpy as np
import pytest

from oracle import bf16_to_f64, moe, mxfp4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import bit_weight_quantized_amd as qmm  # noqa: E402
from test_gpu_moe_layer import CASES, DEV, F32, M, Layer, bf16_bits, dev, guarded, say  # noqa: E402
from test_gpu_mxfp4 import _check_guards, _gpu  # noqa: E402,F401


class Half(Layer):
    more = 0

    def buffers(self):
        return {**super().buffers(), "ws": guarded((2 * self.t * self.k * self.inter + self.more,), 0xFF, torch.uint8)}

    def check(self, o, clear_share=0.9):
        with mock.patch.object(moe, "layer", functools.partial(moe.layer, kept=moe.pairs)):
            super().check(o, clear_share)


@pytest.mark.parametrize("case", CASES)
def test_layer(case):
    say("moe layer, half", case)
    l = Half(case, 8000 + case[0] + case[1] + case[3], pad=256 * (case[0] % 3))
    l.more = 16 * (case[1] % 2)
    l.check(l.run())


@pytest.mark.parametrize("t", [1, 4, 5, 8, 9, 16])
def test_every_token_to_one_expert(t):
    l = Half((t, 7, 1, 672, 352, "softmax", False, 1, 1, False, True, F32, 0, True), 8100 + t)
    l.logits[:] = 0.0
    l.logits[:, 5] = 1.0
    l.check(l.run())


#      long axes, wide outputs in several rounds, the most experts and pairs
@pytest.mark.parametrize("t,ne,k,d,inter", [(2, 3, 2, 32, 65536), (1, 2, 2, 20000, 96), (16, 1024, 16, 32, 32),
                                            (4, 80, 64, 64, 32), (16, 2, 2, 64, 8224)])
def test_limits(t, ne, k, d, inter):
    say("half, limits", t, ne, k, d, inter)
    l = Half((t, ne, k, d, inter, "softmax", False, 1, 1, False, True, F32, 0, True), 9600 + t)
    l.check(l.run())


def test_tokens_with_few_experts_or_none_left():
    l = Half((11, 30, 6, 352, 192, "sigmoid", False, 1, 1, False, True, F32, 0, True), 8200)
    rng = np.random.default_rng(8201)
    for i in range(11):
        row = np.full(30, -np.inf)
        left = rng.choice(30, min(i, 8), replace=False)
        row[left] = l.logits[i, left]
        l.logits[i] = row
    o = l.run()
    assert np.all(o["topk"].cpu().numpy()[0] == -1)
    l.check(o)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_bad_activations_stay_in_their_token(bad):
    l = Half((9, 6, 3, 416, 224, "softmax", False, 1, 1, False, True, F32, 0, False), 8500)
    good = l.run()
    l.x[4, 77] = bf16_bits(np.array([bad]))[0]
    o = l.run()
    keep = [i for i in range(9) if i != 4]
    assert torch.equal(o["out"][keep], good["out"][keep])
    assert not bool(torch.isfinite(o["out"][4].float()).any())


def test_the_largest_activations():
    """gate and up near 2^63: h is near bf16's largest, beside it and past it, of either sign."""
    l = Half((4, 2, 2, 64, 32, "softmax", False, 1, 1, False, True, F32, 0, False), 9800)
    l.gate_up.zero_()
    one = torch.full((64, 32), 0x22, dtype=torch.uint8, device=DEV)         # every code 1
    up = one.clone()
    up[32:] = 0xAA                                                           # up rows -1
    for e in range(2):
        qmm.qmm_pack(M, 64, 64, up if e else one, torch.full((64, 2), 127, dtype=torch.uint8, device=DEV), None, l.gate_up[e])
        qmm.qmm_pack(M, 64, 32, one[:, :16].contiguous(), torch.full((64, 1), 27, dtype=torch.uint8, device=DEV), None, l.down[e])
    x = np.zeros((4, 64), np.float32)
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 2.0 ** 63, 1.99 * 2.0 ** 63, 2.0 ** 64, 2.0 ** 64
    l.x = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
    for e, sign in ((0, 1.0), (1, -1.0)):
        l.logits[:] = -np.inf
        l.logits[:, e] = 0.0
        out = sign * l.run()["out"].float()
        assert bool((out[0] == 2.0 ** 126 * 32 * 2.0 ** -100 * 2.5).all())
        v = float(torch.tensor(1.99).bfloat16())
        assert bool(((out[1] - v * v * 2.0 ** 126 * 32 * 2.0 ** -100 * 2.5).abs() <= 2.0 ** -8 * out[1]).all())
        assert bool((out[2:] == np.inf).all())                               # 2^128


@pytest.mark.parametrize("kind", [Half, Layer])
def test_numbers_that_round_to_infinity(kind):
    """h = 2^128 - 2^114, a finite fp32 past bf16's largest: infinite, not NaN, of either sign."""
    l = kind((2, 2, 1, 64, 32, "softmax", False, 1, 1, False, True, F32, 0, False), 9810)
    for e, minus in ((0, 0), (1, 8)):
        c = np.zeros((64, 64), np.int64)
        c[:32, :2] = 2                                         # gate: x0 + x1
        c[32:, 2] = 2 + minus                                  # up: x2 or -x2
        qmm.qmm_pack(M, 64, 64, dev(mxfp4.pack_codes(c)), dev(np.full((64, 2), 127, np.uint8)), None, l.gate_up[e])
        ones = dev(np.full((64, 16), 0x22, np.uint8))
        qmm.qmm_pack(M, 64, 32, ones, dev(np.full((64, 1), 27, np.uint8)), None, l.down[e])
    x = np.zeros((2, 64), np.float32)
    x[:, 0], x[:, 1], x[:, 2] = 2.0 ** 63 * (2 - 2.0 ** -7), 2.0 ** 63 * (2.0 ** -7 - 2.0 ** -13), 2.0 ** 64
    l.x = bf16_bits(x)
    l.logits = np.array([[1.0, -1.0], [-1.0, 1.0]])
    out = l.run()["out"].float()
    assert bool((out[0] == np.inf).all()) and bool((out[1] == -np.inf).all())


def far_pairs(kind, seed, tokens):
    """A layer whose h is silu(g)·c·2^e with c and e of each output's own, far apart, and whose down
    matrix takes single outputs and sums; shared takes out what bf16 leaves of them."""
    d = inter = 64
    l = kind((tokens, 1, 1, d, inter, "softmax", False, 1, 1, False, True, F32, 0, True), seed)
    l.scale = 1.0
    rng = np.random.default_rng(seed)
    gate, up = np.zeros((2, inter, d), np.int64)
    gate[:, 0] = 2                                             # 1
    up[:, 1] = rng.choice([1, 2, 3, 4, 5, 6, 7, 9, 15], inter)
    e = np.full((2 * inter, d // 32), 127)
    e[inter:] = rng.integers(107, 148, (inter, 1))
    down = np.zeros((d, inter), np.int64)
    down[np.arange(d), np.arange(d)] = 2
    down[:, rng.integers(0, inter, 3)] = 10                    # and three of them subtracted
    for rows, codes, exps, into, blob in ((2 * inter, np.concatenate([gate, up]), e, l.gu, l.gate_up),
                                          (d, down, np.full((d, inter // 32), 127), l.dn, l.down)):
        q, x = mxfp4.pack_codes(codes), exps.astype(np.uint8)
        qmm.qmm_pack(M, rows, 64, dev(q), dev(x), None, blob[0])
        into[0] = mxfp4.dequant(q, x)
    l.x = bf16_bits(rng.normal(0, 1, (tokens, d)) + np.r_[3.0, np.zeros(d - 1)])
    g, u = np.split(bf16_to_f64(l.x) @ l.gu[0].T, 2, 1)
    l.shared = bf16_bits(-(mxfp4.silu(g) * u) @ l.dn[0].T)
    return l


@pytest.mark.parametrize("tokens", [1, 3, 6, 13])
def test_neighbours_far_apart(tokens):
    for kind in (Half, Layer):
        l = far_pairs(kind, 9900 + tokens, tokens)
        l.check(l.run())


def test_subnormal_and_zero_activations():
    """h down to fp32's smallest, at most half of the least unit off (seen 2^100 times larger)."""
    l = far_pairs(Half, 9950, 5)
    l.shared = None
    up = np.zeros((64, 64), np.int64)
    up[:, 1] = 2
    rng = np.random.default_rng(9951)
    e = np.full((128, 2), 127)
    e[64:] = rng.integers(2, 14, (64, 1))
    codes = np.concatenate([np.where(np.arange(64) == 0, 2, 0) * np.ones((64, 1), np.int64), up])
    codes[70:74] = 0                                           # h of 0
    q, x = mxfp4.pack_codes(codes), e.astype(np.uint8)
    qmm.qmm_pack(M, 128, 64, dev(q), dev(x), None, l.gate_up[0])
    l.gu[0] = mxfp4.dequant(q, x)
    q, x = mxfp4.pack_codes(2 * np.eye(64, dtype=np.int64)), np.full((64, 2), 227, np.uint8)
    qmm.qmm_pack(M, 64, 64, dev(q), dev(x), None, l.down[0])
    l.dn[0] = mxfp4.dequant(q, x)
    o = l.run()
    l.check(o)
    assert np.all(o["out"].float().cpu().numpy()[:, 6:10] == 0)


def test_graph_replays_follow_the_inputs_beside_whole_workspaces():
    """A captured call in half, one in the whole workspace on another stream; each replay equals
    its own eager call."""
    case = (6, 14, 3, 480, 256, "softmax", False, 1, 1, False, True, F32, 0, True)
    both = [Half(case, 8900), Layer(case, 8900)]
    ins, outs, graphs = [l.inputs() for l in both], [l.buffers() for l in both], []
    for l, i, o in zip(both, ins, outs):
        l.call(i, o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            l.call(i, o)
        graphs.append(g)
    rng = np.random.default_rng(8901)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in range(4):
        logits, x = rng.integers(-200, 200, (6, 14)) / 64.0, bf16_bits(rng.normal(0, 1, (6, 480)))
        for l, i, o in zip(both, ins, outs):
            l.logits, l.x = logits, x
            fresh = l.inputs()
            i["logits"].copy_(fresh["logits"])
            i["x"].copy_(fresh["x"])
            for key in ("topk", "weights", "out", "ws"):
                o[key].fill_(3)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for l, o in zip(both, outs):
            want = l.run()
            for key in ("topk", "weights", "out"):
                assert torch.equal(o[key], want[key]), (r, key)
            l.check(o)
