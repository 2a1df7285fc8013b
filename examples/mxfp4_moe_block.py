"""The experts of a mixture-of-experts layer on one set of packed MXFP4 weights, both ways that
a server needs them:

  prompts        qmm_route_topk                  logits -> choices, weights, segment tables
                 qmm_mxfp4_quant                 activations to 4 bits
                 qmm_mxfp4_grouped_gemm_swiglu   gate_up with SwiGLU, quantised again
                 qmm_mxfp4_grouped_gemm          down
                 qmm_moe_gather                  weighted sum per token
  up to 16       qmm_moe_layer                   all of it in two launches, activations bf16
  tokens

Every buffer is allocated once; a pass launches kernels only, so it can be captured into a
graph.  Weights are random.

  python examples/mxfp4_moe_block.py [--tokens N] [--dim D] [--inter I] [--experts E] [--top-k K]

checks both against the same experts in fp32 and prints their times.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_quantized_amd as qmm  # noqa: E402

M, FIT, F32 = qmm.QMM_MXFP4_G32, qmm.QMM_MX_FIT, qmm.QMM_F32
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
FEW = 16


def quantize(w: torch.Tensor):
    """bf16 [n, d] -> codes and exponents, the blocks' maxima fitted, by the library's own call."""
    n, d = w.shape
    codes = torch.empty(n, d // 2, dtype=torch.uint8, device=w.device)
    e8m0 = torch.empty(n, qmm.qmm_mxfp4_scale_bytes(d), dtype=torch.uint8, device=w.device)
    qmm.qmm_mxfp4_quant(w, n, d, d, FIT, codes, e8m0)
    return codes, e8m0[:, :d // 32].contiguous()


def dequantize(codes: torch.Tensor, e8m0: torch.Tensor) -> torch.Tensor:
    v = VALUES.to(codes.device)[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(e8m0.float() - 127.0)[..., None]).flatten(-2)


class Mxfp4Experts:
    """Calls of at most `tokens` tokens."""

    def __init__(self, tokens, dim, inter, experts, top_k, seed=0, device="cuda"):
        self.d, self.i, self.e, self.k = dim, inter, experts, top_k
        g = torch.Generator(device=device).manual_seed(seed)

        def stack(n, d):
            plain, blobs = [], torch.empty(experts, qmm.qmm_packed_bytes(M, n, d), dtype=torch.uint8, device=device)
            for e in range(experts):
                codes, e8m0 = quantize((torch.randn(n, d, generator=g, device=device) * d ** -0.5).bfloat16())
                qmm.qmm_pack(M, n, d, codes, e8m0, None, blobs[e])
                plain.append(dequantize(codes, e8m0))
            return plain, blobs

        self.plain_gu, self.gu = stack(2 * inter, dim)
        self.plain_down, self.down = stack(dim, inter)

        def empty(*shape, dtype):
            return torch.empty(*shape, dtype=dtype, device=device)

        m, i32, u8, bf = tokens * top_k, torch.int32, torch.uint8, torch.bfloat16
        self.topk, self.weights = empty(tokens, top_k, dtype=i32), empty(tokens, top_k, dtype=torch.float32)
        self.seg_expert, self.seg_offsets = empty(experts, dtype=i32), empty(experts + 1, dtype=i32)
        self.row_index, self.slot_row = empty(m, dtype=i32), empty(tokens, top_k, dtype=i32)
        self.xq, self.xs = empty(tokens, dim // 2, dtype=u8), empty(tokens, qmm.qmm_mxfp4_scale_bytes(dim), dtype=u8)
        self.hq, self.hs = empty(m, inter // 2, dtype=u8), empty(m, qmm.qmm_mxfp4_scale_bytes(inter), dtype=u8)
        self.o, self.out = empty(m, dim, dtype=bf), empty(tokens, dim, dtype=bf)
        route, few = qmm.qmm_route_topk_workspace_bytes(tokens, experts), min(tokens, FEW, 256 // top_k)
        self.ws = empty(max(route, qmm.qmm_moe_layer_workspace_bytes(few, top_k, inter)), dtype=u8)

    def few(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        t = x.shape[0]
        qmm.qmm_moe_layer(M, self.gu, self.gu.shape[1], self.down, self.down.shape[1], self.e, self.d, self.i, x, t, logits,
                          F32, self.e, qmm.QMM_SCORE_SOFTMAX, None, 1, 1, qmm.QMM_GROUP_MAX, self.k, True, 1.0, None,
                          self.topk, self.weights, self.out, self.ws)
        return self.out[:t]

    def many(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        t, d, i, e, k = x.shape[0], self.d, self.i, self.e, self.k
        m = t * k
        qmm.qmm_route_topk(logits, F32, t, e, e, qmm.QMM_SCORE_SOFTMAX, None, 1, 1, qmm.QMM_GROUP_MAX, k, True, 1.0,
                           self.topk, self.weights, self.seg_expert, self.seg_offsets, self.row_index, self.slot_row,
                           self.ws)
        table = (self.seg_expert, self.seg_offsets, e, m, t)
        qmm.qmm_mxfp4_quant(x, t, d, d, FIT, self.xq, self.xs)
        qmm.qmm_mxfp4_grouped_gemm_swiglu(self.gu, self.gu.shape[1], e, 2 * i, d, self.xq, self.xs, t, self.row_index,
                                          *table, FIT, None, self.hq, self.hs)
        qmm.qmm_mxfp4_grouped_gemm(self.down, self.down.shape[1], e, d, i, self.hq, self.hs, m, None, *table, self.o)
        qmm.qmm_moe_gather(self.o, m, d, t, k, self.slot_row, self.weights, None, self.out)
        return self.out[:t]

    def __call__(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """x bf16[t][dim], logits fp32[t][experts]."""
        t = x.shape[0]
        return (self.few if t <= FEW and t * self.k <= 256 else self.many)(x, logits)

    def plain(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        """The same in fp32, activations not quantised."""
        top = torch.topk(logits, self.k)
        weight = torch.softmax(top.values, 1)
        out = torch.zeros(x.shape, device=x.device)
        for e in range(self.e):
            token, slot = torch.nonzero(top.indices == e, as_tuple=True)
            if token.numel():
                gate, up = (x[token].float() @ self.plain_gu[e].T).chunk(2, 1)
                y = torch.nn.functional.silu(gate) * up @ self.plain_down[e].T
                out.index_add_(0, token, y * weight[token, slot, None])
        return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--dim", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--top-k", type=int, default=4)
    a = ap.parse_args(argv)
    block = Mxfp4Experts(a.tokens, a.dim, a.inter, a.experts, a.top_k)
    errors = {}
    for t in sorted({1, min(FEW, a.tokens), a.tokens}):
        g = torch.Generator(device="cuda").manual_seed(t)
        x = torch.randn(t, a.dim, generator=g, device="cuda").bfloat16()
        logits = torch.randn(t, a.experts, generator=g, device="cuda")
        want = block.plain(x, logits)
        out = block(x, logits).float()
        errors[t] = float((out - want).norm() / want.norm())
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(20):
            block(x, logits)
        end.record()
        end.synchronize()
        print(f"{t} tokens: relative error {errors[t]:.4f}, {start.elapsed_time(end) / 20 * 1e3:.1f} us a pass")
    return errors


if __name__ == "__main__":
    main()
