"""A mixture-of-experts block with block-scaled e4m3 weights, from one residual
stream to the next, on the library's calls:

  qmm_norm_residual            h = rms(v)·w, as bf16 (router) and codes (experts)
  h·Wrᵀ (torch)                router logits
  qmm_route_topk               scores, groups, top-k, weights and segment tables
  qmm_fp8_grouped_gemm_swiglu  routed experts: gate_up with SwiGLU on the codes of h
  qmm_fp8_quant                their outputs as codes
  qmm_fp8_grouped_gemm         routed experts: down
  (the same three              the shared expert, as one segment of all tokens)
  qmm_moe_gather               weighted sum per token, plus the shared expert
  qmm_norm_residual            v + rms(out)·w', and the next block's h

Every buffer is allocated once; a forward pass launches kernels only, so it can be
captured into a graph.  Weights are random.

  python examples/fp8_moe_block.py [--tokens N] [--dim D] [--inter I] [--experts E] [--top-k K]

checks a pass against the same block in fp32 and prints its time.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_quantized_amd as qmm  # noqa: E402

BLOCK = 128
EPS = 1e-6


def quantize_weights(w: torch.Tensor):
    """[..., n, d] -> e4m3 codes (uint8) and fp32 scales [..., ceil(n/128), ceil(d/128)], amax / 448 a block."""
    n, d = w.shape[-2:]
    nb, db = -(-n // BLOCK), -(-d // BLOCK)
    p = torch.nn.functional.pad(w.float(), (0, db * BLOCK - d, 0, nb * BLOCK - n))
    p = p.unflatten(-1, (db, BLOCK)).unflatten(-3, (nb, BLOCK))          # [..., nb, 128, db, 128]
    scales = (p.abs().amax((-3, -1)) / 448.0).clamp_min(1e-20)
    q = (p / scales[..., :, None, :, None]).flatten(-2).flatten(-3, -2)[..., :n, :d]
    return q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), scales.contiguous()


def dequantize(q: torch.Tensor, scales: torch.Tensor, rows: int = BLOCK) -> torch.Tensor:
    """Codes and scales (a block of `rows` by 128) -> fp32."""
    n, d = q.shape[-2:]
    s = scales.repeat_interleave(rows, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :d]
    return q.view(torch.float8_e4m3fn).float() * s


class Fp8MoeBlock:
    def __init__(self, tokens, dim, inter, experts, top_k, groups=1, keep_groups=1, scale=1.0, seed=0, device="cuda"):
        self.t, self.d, self.i, self.e, self.k = tokens, dim, inter, experts, top_k
        self.groups, self.keep, self.scale = groups, keep_groups, scale
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std=1.0):
            return torch.randn(*shape, generator=g, device=device) * std

        def gate_up(n_experts):   # each half has scale rows of its own
            halves = [quantize_weights(randn(n_experts, inter, dim, std=dim ** -0.5)) for _ in range(2)]
            return torch.cat([h[0] for h in halves], 1), torch.cat([h[1] for h in halves], 1)

        self.gu, self.gu_s = gate_up(experts)
        self.down, self.down_s = quantize_weights(randn(experts, dim, inter, std=inter ** -0.5))
        self.sgu, self.sgu_s = gate_up(1)
        self.sdown, self.sdown_s = quantize_weights(randn(1, dim, inter, std=inter ** -0.5))
        self.router = randn(experts, dim, std=dim ** -0.5)
        self.bias = randn(experts, std=0.01)
        self.pre_w, self.post_w, self.next_w = ((1 + randn(dim, std=0.1)).bfloat16() for _ in range(3))

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=device)

        m = tokens * top_k
        i32, f32, u8 = torch.int32, torch.float32, torch.uint8
        nb, ib = -(-dim // BLOCK), -(-inter // BLOCK)
        self.h, self.hq, self.hs = empty(tokens, dim), empty(tokens, dim, dtype=u8), empty(tokens, nb, dtype=f32)
        self.topk, self.weights = empty(tokens, top_k, dtype=i32), empty(tokens, top_k, dtype=f32)
        self.slot_row = empty(tokens, top_k, dtype=i32)
        self.seg_expert, self.seg_offsets = empty(experts, dtype=i32), empty(experts + 1, dtype=i32)
        self.row_index = empty(m, dtype=i32)
        ws = qmm.qmm_route_topk_workspace_bytes(tokens, experts)
        self.ws = empty(max(ws, 4), dtype=u8)
        self.act, self.act_q, self.act_s = empty(m, inter), empty(m, inter, dtype=u8), empty(m, ib, dtype=f32)
        self.o = empty(m, dim)
        self.sact, self.sact_q, self.sact_s = empty(tokens, inter), empty(tokens, inter, dtype=u8), empty(tokens, ib, dtype=f32)
        self.shared, self.out = empty(tokens, dim), empty(tokens, dim)
        self.r_out, self.next_h = empty(tokens, dim), empty(tokens, dim)
        self.one_seg = torch.zeros(1, dtype=i32, device=device)
        self.one_off = torch.tensor([0, tokens], dtype=i32, device=device)

    def __call__(self, r: torch.Tensor):
        """r bf16[t][d] -> the residual after the block and the next block's normed input."""
        t, d, i, e, k = self.t, self.d, self.i, self.e, self.k
        bf16 = qmm.QMM_BF16
        # no block before this one: v = r, h = rms(v)·pre_w
        qmm.qmm_norm_residual(t, d, None, 0, None, None, 0, 1, r, bf16, d, 1.0, None, 0, self.pre_w, 0.0, EPS,
                              self.h, d, self.hq, self.hs)
        logits = self.h.float() @ self.router.T
        qmm.qmm_route_topk(logits, qmm.QMM_F32, t, e, e, qmm.QMM_SCORE_SIGMOID, self.bias, self.groups, self.keep,
                           qmm.QMM_GROUP_TOP2, k, 1, self.scale, self.topk, self.weights, self.seg_expert,
                           self.seg_offsets, self.row_index, self.slot_row, self.ws)
        m = t * k
        table = (self.seg_expert, self.seg_offsets, e, m, t)
        qmm.qmm_fp8_grouped_gemm_swiglu(self.gu, self.gu_s, e, 2 * i, d, self.hq, self.hs, t, self.row_index, *table, self.act)
        qmm.qmm_fp8_quant(self.act, m, i, i, self.act_q, self.act_s)
        qmm.qmm_fp8_grouped_gemm(self.down, self.down_s, e, d, i, self.act_q, self.act_s, m, None, *table, self.o)
        one = (self.one_seg, self.one_off, 1, t, t)
        qmm.qmm_fp8_grouped_gemm_swiglu(self.sgu, self.sgu_s, 1, 2 * i, d, self.hq, self.hs, t, None, *one, self.sact)
        qmm.qmm_fp8_quant(self.sact, t, i, i, self.sact_q, self.sact_s)
        qmm.qmm_fp8_gemm(self.sdown, self.sdown_s, t, d, i, self.sact_q, self.sact_s, self.shared, d)
        qmm.qmm_moe_gather(self.o, m, d, t, k, self.slot_row, self.weights, self.shared, self.out)
        # v = r + rms(out)·post_w, next h = rms(v)·next_w
        qmm.qmm_norm_residual(t, d, self.out, d, self.post_w, None, 0, 1, r, bf16, d, 1.0, self.r_out, d, self.next_w,
                              0.0, EPS, self.next_h, d, None, None)
        return self.r_out, self.next_h

    def plain(self, r: torch.Tensor):
        """The block in fp32, on the experts that the last pass chose and the codes that its norm gave."""
        def rms(v, w):
            return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()

        def expert(x, gu, gu_s, down, down_s):
            half = gu_s.shape[0] // 2
            gate, up = (dequantize(gu[a * self.i:(a + 1) * self.i], gu_s[a * half:(a + 1) * half]) for a in (0, 1))
            return torch.nn.functional.silu(x @ gate.T) * (x @ up.T) @ dequantize(down, down_s).T

        v = r.float()
        x = dequantize(self.hq, self.hs, rows=1)
        out = expert(x, self.sgu[0], self.sgu_s[0], self.sdown[0], self.sdown_s[0])
        p = torch.sigmoid(rms(v, self.pre_w).bfloat16().float() @ self.router.T)
        chosen = p.gather(1, self.topk.long())
        weight = chosen / chosen.sum(1, keepdim=True) * self.scale
        for e in range(self.e):
            token, slot = torch.nonzero(self.topk == e, as_tuple=True)
            if token.numel():
                y = expert(x[token], self.gu[e], self.gu_s[e], self.down[e], self.down_s[e])
                out.index_add_(0, token, y * weight[token, slot, None])
        v = v + rms(out, self.post_w)
        return v, rms(v, self.next_w)


def main(argv=None) -> float:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--dim", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1408)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=6)
    ap.add_argument("--groups", type=int, default=8)
    ap.add_argument("--keep-groups", type=int, default=4)
    ap.add_argument("--repeat", type=int, default=50)
    a = ap.parse_args(argv)
    block = Fp8MoeBlock(a.tokens, a.dim, a.inter, a.experts, a.top_k, a.groups, a.keep_groups, scale=2.5)
    r = torch.randn(a.tokens, a.dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    got = [x.float() for x in block(r)]
    far = max(float((g - w).norm() / w.norm()) for g, w in zip(got, block.plain(r)))
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.repeat):
        block(r)
    stop.record()
    stop.synchronize()
    us = start.elapsed_time(stop) * 1e3 / max(a.repeat, 1)
    print(f"{a.tokens} tokens x {a.dim}, top {a.top_k} of {a.experts} experts of {a.inter}: "
          f"{us:.1f} us a block, relative difference from fp32 {far:.4f}")
    return far


if __name__ == "__main__":
    main()
