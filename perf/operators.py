"""Cases that measure the 8-bit expert path: block-scaled e4m3 products, the quantiser
that feeds them, the grouped top-k router and the norms around a block.

``own = False`` computes each operator in its plain form with elementary torch
operations in 32 bits; ``own = True`` makes the library's calls.  Both take the same
state from ``prepare``: inputs and weights in the layouts of ``include/qmm.h``.

Formulas (b: blocks of 128 along the reduction axis, nb of them, the last may be short)
  quant    m = max(max_b |x|, 2^-96);  s[t,b] = m / 448,  q = e4m3(x * f) with f = 448 / m and
           x * f fp32 numbers: bf16 values of a block often lie midway between two codes,
           so the roundings before the last one belong to the definition
  gemm     y[t,n] = sum_b xs[t,b] * ws[n/128,b] * sum_{k in b} xq[t,k] * wq[n,k]
  experts  per routed row: h = silu(x G^T) * (x U^T) on quantised x, then quantised h
           times the down matrix; out[t] = sum_j weight[t,j] * o[row of slot j]
  route    s = softmax(l) or sigmoid(l); groups ranked by the best or the sum of the two
           best s + bias; the k best experts of the kept groups; weights renormalised
  norm     v = a*r + gate * rms(o)*w1;  h = rms(v)*w2;  h also as e4m3 with its scales (of h before it is rounded)
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3 = torch.float8_e4m3fn
FLOOR = 2.0 ** -96     # smallest block maximum that scales are made from
BF16, F32 = 1, 2       # the library's type codes
SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


def blocks(d):
    return -(-d // BLOCK)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode token against a wide projection: the weights' bytes are the whole cost
        {"name": "gemm_decode", "op": "gemm", "t": 1, "n": 13824, "d": 5120},
        # an odd decode batch on the narrower way back
        {"name": "gemm_batch", "op": "gemm", "t": 37, "n": 5120, "d": 13824},
        # a short ragged prompt: no size is a multiple of a tile, the last block is short
        {"name": "gemm_ragged", "op": "gemm", "t": 333, "n": 1000, "d": 2064},
        # prefill: the matrix cores' rate is the whole cost
        {"name": "gemm_prefill", "op": "gemm", "t": 2048, "n": 13824, "d": 5120},
        # four decode tokens through routed experts: nearly every row has its own expert
        {"name": "experts_decode", "op": "experts", "t": 4, "experts": 128, "k": 8, "d": 3584, "inter": 2048},
        # routed prefill: hundreds of rows an expert
        {"name": "experts_prefill", "op": "experts", "t": 4096, "experts": 64, "k": 8, "d": 3584, "inter": 2048},
        # the activations of a decode batch: launch latency
        {"name": "quant_decode", "op": "quant", "t": 16, "d": 3584},
        # the activations of a prefill of a wide projection: memory bandwidth
        {"name": "quant_prefill", "op": "quant", "t": 8192, "d": 13824},
        # one decode token, sigmoid scores with a balance bias and expert groups: latency
        {"name": "route_decode", "op": "route", "t": 1, "experts": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "by": "top2", "renorm": True, "scale": 2.5, "logits": "f32", "masked": 0.0},
        # the same router over a long prefill, logits in bf16 (many exact ties)
        {"name": "route_prefill", "op": "route", "t": 16384, "experts": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "by": "top2", "renorm": True, "scale": 2.5, "logits": "bf16", "masked": 0.0},
        # one decode token between two blocks: latency
        {"name": "norm_decode", "op": "norm", "t": 1, "d": 5120, "residual": "bf16", "post": True, "gate_rows": 1,
         "out": "both", "offset": 0.0},
        # prefill between two blocks, one gate row for each sequence of 2048 tokens
        {"name": "norm_prefill", "op": "norm", "t": 8192, "d": 5120, "residual": "bf16", "post": True,
         "gate_rows": 2048, "out": "both", "offset": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "experts", "experts", "quant", "route", "norm"])
    if op == "gemm":
        while True:
            c = {"op": op, "t": _log(rng, 1, 4096), "n": _log(rng, 64, 14336), "d": 16 * _log(rng, 8, 1024)}
            if c["t"] * c["n"] * c["d"] <= 2048 * 13824 * 5120 and c["n"] * c["d"] >= 1 << 17:
                return c
    if op == "experts":
        while True:
            c = {"op": op, "t": _log(rng, 1, 4096), "experts": rng.choice([8, 16, 60, 64, 128]), "k": rng.randint(1, 8),
                 "d": 16 * _log(rng, 32, 256), "inter": 16 * _log(rng, 16, 128)}
            if (c["t"] * c["k"] * c["d"] * c["inter"] <= 4096 * 8 * 3584 * 2048
                    and c["experts"] * c["d"] * c["inter"] <= 64 * 3584 * 2048):
                return c
    if op == "quant":
        return {"op": op, "t": _log(rng, 1, 8192), "d": 16 * _log(rng, 8, 864)}
    if op == "route":
        experts, groups = rng.choice([(8, 1), (60, 1), (64, 8), (128, 1), (160, 8), (256, 8), (384, 1), (384, 12), (896, 1)])
        score = rng.choice(["softmax", "sigmoid"])
        # softmax scores are ranked by the logits themselves where no bias is added
        return {"op": op, "t": _log(rng, 1, 16384), "experts": experts, "k": rng.randint(1, 8), "score": score,
                "bias": score == "sigmoid" and rng.random() < 0.7, "groups": groups,
                "keep": max(1, groups // 2), "by": "max" if score == "softmax" else rng.choice(["max", "top2"]),
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "logits": rng.choice(["f32", "bf16"]),
                "masked": rng.choice([0.0, 0.3])}
    return {"op": op, "t": _log(rng, 1, 8192), "d": 16 * _log(rng, 8, 512), "residual": rng.choice(["bf16", "f32"]),
            "post": rng.random() < 0.8, "gate_rows": rng.choice([0, 1, 100000]),
            "out": rng.choice(["bf16", "fp8", "both"]), "offset": rng.choice([0.0, 1.0])}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFFFFFF)


def _activations(g, t, d):
    """bf16 rows as a norm leaves them: near normal, a few channels much larger."""
    x = torch.randn(t, d, generator=g, device=DEV)
    wide = (torch.rand(d, generator=g, device=DEV) < 0.004).float() * 12.0 + 1.0
    return (x * wide).to(torch.bfloat16)


def _weights(g, n, d):
    """e4m3 codes of normal weights and one fp32 scale for each block of 128 x 128."""
    q = torch.randn(n, d, generator=g, device=DEV).clamp_(-4.0, 4.0).mul_(112.0).to(E4M3)
    s = (0.5 + torch.rand(blocks(n), blocks(d), generator=g, device=DEV)) * (0.02 / 112.0)
    return q, s


def _expert_weights(g, experts, n, d, halves):
    """A stack of expert matrices; `halves`: gate rows, then up rows, each with blocks of its own."""
    q = torch.empty(experts, n, d, dtype=E4M3, device=DEV)
    for e in range(experts):
        q[e] = torch.randn(n, d, generator=g, device=DEV).clamp_(-4.0, 4.0).mul_(112.0).to(E4M3)
    nbn = halves * blocks(n // halves)
    s = (0.5 + torch.rand(experts, nbn, blocks(d), generator=g, device=DEV)) * (0.02 / 112.0)
    return q, s


def _routing(g, t, experts, k):
    """k distinct experts a token (some experts more popular), weights, and the grouped order."""
    like = torch.rand(t, experts, generator=g, device=DEV) + 0.3 * torch.rand(experts, generator=g, device=DEV)
    ids = like.topk(k, dim=1).indices
    w = torch.rand(t, k, generator=g, device=DEV) + 0.1
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(flat, minlength=experts).cumsum(0)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(t * k, device=DEV)
    return {"weights": w / w.sum(1, keepdim=True), "seg_expert": torch.arange(experts, dtype=torch.int32, device=DEV),
            "seg_offsets": offsets, "row_index": (order // k).to(torch.int32),
            "slot_row": slot.reshape(t, k).to(torch.int32)}


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c}
    if c["op"] == "gemm":
        t, n, d = c["t"], c["n"], c["d"]
        s["x"], s["xs"] = _quant_plain(_activations(g, t, d))
        s["w"], s["ws"] = _weights(g, n, d)
        s["y"] = torch.empty(t, n, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "experts":
        t, e, k, d, i = c["t"], c["experts"], c["k"], c["d"], c["inter"]
        s["x"] = _activations(g, t, d)
        s["gu"], s["gus"] = _expert_weights(g, e, 2 * i, d, 2)
        s["dn"], s["dns"] = _expert_weights(g, e, d, i, 1)
        s |= _routing(g, t, e, k)
        s["most"] = int((s["seg_offsets"][1:] - s["seg_offsets"][:-1]).max())
        m = t * k
        s["xq"] = torch.empty(t, d, dtype=torch.uint8, device=DEV)
        s["xs"] = torch.empty(t, blocks(d), device=DEV)
        s["h"] = torch.empty(m, i, dtype=torch.bfloat16, device=DEV)
        s["hq"] = torch.empty(m, i, dtype=torch.uint8, device=DEV)
        s["hs"] = torch.empty(m, blocks(i), device=DEV)
        s["o"] = torch.empty(m, d, dtype=torch.bfloat16, device=DEV)
        s["out"] = torch.empty(t, d, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "quant":
        t, d = c["t"], c["d"]
        s["x"] = _activations(g, t, d)
        s["q"] = torch.empty(t, d, dtype=torch.uint8, device=DEV)
        s["s"] = torch.empty(t, blocks(d), device=DEV)
    elif c["op"] == "route":
        t, e, k = c["t"], c["experts"], c["k"]
        l = torch.randn(t, e, generator=g, device=DEV) * 1.5 + 0.5 * torch.randn(e, generator=g, device=DEV)
        if c["masked"]:
            l[torch.rand(t, e, generator=g, device=DEV) < c["masked"]] = -math.inf
            l[torch.rand(t, generator=g, device=DEV) < 0.05] = -math.inf     # a token with nothing left
        s["l"] = l if c["logits"] == "f32" else l.to(torch.bfloat16)
        s["bias"] = 0.1 * torch.randn(e, generator=g, device=DEV) if c["bias"] else None
        s["topk"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(t, k, device=DEV)
        s["seg_expert"] = torch.empty(e, dtype=torch.int32, device=DEV)
        s["seg_offsets"] = torch.empty(e + 1, dtype=torch.int32, device=DEV)
        s["row_index"] = torch.empty(t * k, dtype=torch.int32, device=DEV)
        s["slot_row"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
        # as much as the router's work space takes at most: two tables of e counts for every 32 tokens
        s["ws"] = torch.empty(8 * (e + 1) * (-(-t // 32) + 1), dtype=torch.uint8, device=DEV)
    else:
        t, d = c["t"], c["d"]
        s["o"] = _activations(g, t, d)
        rt = torch.bfloat16 if c["residual"] == "bf16" else torch.float32
        s["r"] = (3.0 * torch.randn(t, d, generator=g, device=DEV)).to(rt)
        near = 0.0 if c["offset"] else 1.0
        w = lambda: (near + 0.2 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)  # noqa: E731
        s["w1"] = w() if c["post"] else None
        s["w2"] = w()
        rows = -(-t // c["gate_rows"]) if c["gate_rows"] else 0
        s["gate"] = (0.5 * torch.randn(rows, d, generator=g, device=DEV)).to(torch.bfloat16) if rows else None
        s["scale"], s["eps"] = 0.75, 1e-6
        s["v"] = torch.empty(t, d, dtype=rt, device=DEV)
        s["h"] = torch.empty(t, d, dtype=torch.bfloat16, device=DEV) if c["out"] != "fp8" else None
        s["q"] = torch.empty(t, d, dtype=torch.uint8, device=DEV) if c["out"] != "bf16" else None
        s["s"] = torch.empty(t, blocks(d), device=DEV) if c["out"] != "bf16" else None
    return s


# ---------------------------------------------------------------- plain forms

def _pad(x):
    d = x.shape[-1]
    return torch.nn.functional.pad(x, (0, blocks(d) * BLOCK - d))


def _quant_plain(x):
    d = x.shape[-1]
    b = _pad(x.float()).unflatten(-1, (-1, BLOCK))
    most = b.abs().amax(-1).clamp_min(FLOOR)
    factor = torch.full_like(most, 448.0) / most      # one division: a number over a tensor would be a reciprocal times it
    q = (b * factor[..., None]).to(E4M3).flatten(-2)[..., :d]
    return q.contiguous(), most / 448.0


def _spread(s, n, d):
    """Scales of blocks as one factor for each element of the last two axes."""
    return s.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :d]


def _dequant(q, s):
    return q.float() * s.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _gemm_plain(x, xs, w, ws):
    return (_dequant(x, xs) @ (w.float() * _spread(ws, *w.shape)).t()).to(torch.bfloat16)


def _experts_plain(s):
    c, most = s["case"], s["most"]
    e, d, i, m = c["experts"], c["d"], c["inter"], c["t"] * c["k"]
    # the rows of every expert, padded to the longest segment
    at = s["seg_offsets"][:-1, None] + torch.arange(most, device=DEV)
    live = at < s["seg_offsets"][1:, None]
    at = at.clamp_max(m - 1)
    x = _dequant(*_quant_plain(s["x"]))[s["row_index"][at]]
    gu = s["gu"].float()
    gu[:, :i] *= _spread(s["gus"][:, :blocks(i)], i, d)
    gu[:, i:] *= _spread(s["gus"][:, blocks(i):], i, d)
    y = torch.bmm(gu, x.transpose(1, 2).contiguous())
    del gu, x
    h = (y[:, :i] / (1.0 + torch.exp(-y[:, :i])) * y[:, i:]).to(torch.bfloat16)
    h = _dequant(*_quant_plain(h.transpose(1, 2)))
    o = torch.bmm(s["dn"].float() * _spread(s["dns"], d, i), h.transpose(1, 2).contiguous())
    o = o.transpose(1, 2)[live].to(torch.bfloat16)          # grouped order again
    return (o[s["slot_row"]].float() * s["weights"][..., None]).sum(1).to(torch.bfloat16)


def _route_plain(s):
    c = s["case"]
    t, e, k = c["t"], c["experts"], c["k"]
    l = s["l"].float()
    dead = l == -math.inf
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
        rank = p
    else:
        z = torch.exp(l - l.amax(1, keepdim=True))
        p = (z / z.sum(1, keepdim=True)).masked_fill(dead, 0.0)
        rank = l
    if s["bias"] is not None:
        rank = p + s["bias"]
    rank = rank.masked_fill(dead, -math.inf)
    if c["groups"] > 1:
        grouped = rank.view(t, c["groups"], -1)
        if c["by"] == "max":
            value = grouped.amax(-1)
        else:
            two = grouped.sort(-1, descending=True).values[..., :2]
            value = two[..., 0] + two[..., 1].masked_fill(two[..., 1] == -math.inf, 0.0)
        kept = value.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
        rank = rank.masked_fill(~keep.repeat_interleave(e // c["groups"], 1), -math.inf)
    best, ids = rank.sort(dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    w = p.gather(1, ids).masked_fill(best == -math.inf, 0.0)
    ids = ids.masked_fill(best == -math.inf, -1)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0.0, w / total, torch.zeros_like(w))
    w = w * c["scale"]
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, e, flat)
    order = key.sort(dim=0, stable=True).indices
    count = torch.zeros(e + 1, dtype=torch.int64, device=DEV).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = count[:e].cumsum(0)
    slot = torch.empty_like(order).scatter_(0, order, torch.arange(t * k, device=DEV))
    rows = (order // k).masked_fill(flat[order] < 0, -1)
    return {"topk": ids.to(torch.int32), "weights": w, "seg_expert": torch.arange(e, dtype=torch.int32, device=DEV),
            "seg_offsets": offsets, "row_index": rows.to(torch.int32),
            "slot_row": slot.masked_fill(flat < 0, -1).view(t, k).to(torch.int32)}


def _norm_plain(s):
    c = s["case"]
    rms = lambda x: x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])  # noqa: E731
    u = s["o"].float()
    if s["w1"] is not None:
        u = rms(u) * (c["offset"] + s["w1"].float())
    if s["gate"] is not None:
        u = u * s["gate"].float()[torch.arange(c["t"], device=DEV) // c["gate_rows"]]
    v = s["scale"] * s["r"].float() + u
    h = rms(v) * (c["offset"] + s["w2"].float())
    got = {"v": v.to(s["r"].dtype)}
    if c["out"] != "fp8":
        got["h"] = h.to(torch.bfloat16)
    if c["out"] != "bf16":
        got["q"], got["s"] = _quant_plain(h)
    return got


# ---------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "gemm":
            return _gemm_plain(s["x"], s["xs"], s["w"], s["ws"])
        if c["op"] == "experts":
            return _experts_plain(s)
        if c["op"] == "quant":
            q, scales = _quant_plain(s["x"])
            return {"q": q, "s": scales}
        return _route_plain(s) if c["op"] == "route" else _norm_plain(s)
    import bit_weight_quantized_amd as qmm
    if c["op"] == "gemm":
        qmm.qmm_fp8_gemm(s["w"], s["ws"], c["t"], c["n"], c["d"], s["x"], s["xs"], s["y"], c["n"])
        return s["y"]
    if c["op"] == "experts":
        t, e, k, d, i = c["t"], c["experts"], c["k"], c["d"], c["inter"]
        m = t * k
        table = (s["seg_expert"], s["seg_offsets"], e, m, t)
        qmm.qmm_fp8_quant(s["x"], t, d, d, s["xq"], s["xs"])
        qmm.qmm_fp8_grouped_gemm_swiglu(s["gu"], s["gus"], e, 2 * i, d, s["xq"], s["xs"], t, s["row_index"], *table, s["h"])
        qmm.qmm_fp8_quant(s["h"], m, i, i, s["hq"], s["hs"])
        qmm.qmm_fp8_grouped_gemm(s["dn"], s["dns"], e, d, i, s["hq"], s["hs"], m, None, *table, s["o"])
        qmm.qmm_moe_gather(s["o"], m, d, t, k, s["slot_row"], s["weights"], None, s["out"])
        return s["out"]
    if c["op"] == "quant":
        qmm.qmm_fp8_quant(s["x"], c["t"], c["d"], c["d"], s["q"], s["s"])
        return {"q": s["q"].view(E4M3), "s": s["s"]}
    if c["op"] == "route":
        t, e, k = c["t"], c["experts"], c["k"]
        qmm.qmm_route_topk(s["l"], BF16 if c["logits"] == "bf16" else F32, t, e, e,
                           SIGMOID if c["score"] == "sigmoid" else SOFTMAX, s["bias"], c["groups"], c["keep"],
                           GROUP_TOP2 if c["by"] == "top2" else GROUP_MAX, k, c["renorm"], c["scale"], s["topk"],
                           s["weights"], s["seg_expert"], s["seg_offsets"], s["row_index"], s["slot_row"], s["ws"])
        return {n: s[n] for n in ("topk", "weights", "seg_expert", "seg_offsets", "row_index", "slot_row")}
    t, d = c["t"], c["d"]
    qmm.qmm_norm_residual(t, d, s["o"], d, s["w1"], s["gate"], d, max(1, c["gate_rows"]), s["r"],
                          BF16 if c["residual"] == "bf16" else F32, d, s["scale"], s["v"], d, s["w2"], c["offset"],
                          s["eps"], s["h"], d, s["q"], s["s"])
    got = {"v": s["v"]}
    if c["out"] != "fp8":
        got["h"] = s["h"]
    if c["out"] != "bf16":
        got["q"], got["s"] = s["q"].view(E4M3), s["s"]
    return got


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "gemm":
        t, n, d = c["t"], c["n"], c["d"]
        return {"bytes": n * d + t * d + 4 * blocks(d) * (blocks(n) + t) + 2 * t * n, "flops": 2 * t * n * d}
    if c["op"] == "experts":
        t, e, k, d, i = c["t"], c["experts"], c["k"], c["d"], c["inter"]
        used = e * (1.0 - (1.0 - k / e) ** t)          # experts that get a row, expected
        return {"bytes": int(used * 3 * i * d) + 4 * t * d + 8 * t * k, "flops": 6 * t * k * i * d}
    if c["op"] == "quant":
        return {"bytes": c["t"] * (3 * c["d"] + 4 * blocks(c["d"])), "flops": 3 * c["t"] * c["d"]}
    if c["op"] == "route":
        t, e, k = c["t"], c["experts"], c["k"]
        return {"bytes": t * e * (4 if c["logits"] == "f32" else 2) + 16 * t * k + 12 * e, "flops": t * e * 8}
    t, d = c["t"], c["d"]
    rows = -(-t // c["gate_rows"]) if c["gate_rows"] else 0
    each = 2 + (4 if c["residual"] == "bf16" else 8) + (2 if c["out"] != "fp8" else 0) + (1 if c["out"] != "bf16" else 0)
    return {"bytes": t * d * each + 2 * d * (1 + c["post"] + rows), "flops": 12 * t * d}


# ---------------------------------------------------------------- the definitions in 64 bits

def _e4m3_64(v):
    """Nearest e4m3 value of a 64-bit number, ties to even: 4 significant bits down to 2^-6, steps of 2^-9 below."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2((torch.frexp(a).exponent - 1).clamp(min=-6).to(torch.float64) - 3.0)
    return torch.copysign(torch.round(a / step) * step, v)


def _quant_64(x):
    """(codes' values, scales) of rows in 64 bits, one block after the other."""
    q, s = torch.empty_like(x), torch.empty(*x.shape[:-1], blocks(x.shape[-1]), dtype=torch.float64, device=x.device)
    for b in range(s.shape[-1]):
        part = x[..., BLOCK * b:BLOCK * (b + 1)]
        most = torch.clamp(part.abs().max(-1).values, min=FLOOR)
        s[..., b] = most / 448.0
        factor = (torch.full_like(most, 448.0) / most).float().double()      # the definition's factor and products are fp32 numbers
        q[..., BLOCK * b:BLOCK * (b + 1)] = _e4m3_64((part * factor[..., None]).float().double())
    return q, s


def _rows_64(q, s):
    v = q.double()
    for b in range(s.shape[-1]):
        v[..., BLOCK * b:BLOCK * (b + 1)] *= s[..., b:b + 1].double()
    return v


def _matrix_64(q, s):
    v = _rows_64(q, s.double().repeat_interleave(BLOCK, 0)[:q.shape[0]])
    return v


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gemm":
        return _rows_64(s["x"], s["xs"]) @ _matrix_64(s["w"], s["ws"]).t()
    if c["op"] == "experts":
        x = _rows_64(*_quant_64(s["x"].double()))
        i, offsets = c["inter"], s["seg_offsets"].tolist()
        out = torch.zeros(c["t"], c["d"], dtype=torch.float64, device=DEV)
        weight = torch.empty(c["t"] * c["k"], dtype=torch.float64, device=DEV)
        weight[s["slot_row"].reshape(-1).long()] = s["weights"].double().reshape(-1)
        for e in range(c["experts"]):
            lo, hi = offsets[e], offsets[e + 1]
            if hi == lo:
                continue
            rows = s["row_index"][lo:hi].long()
            gate = x[rows] @ _matrix_64(s["gu"][e, :i], s["gus"][e, :blocks(i)]).t()
            up = x[rows] @ _matrix_64(s["gu"][e, i:], s["gus"][e, blocks(i):]).t()
            h = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16).double()     # h is held in bf16, then e4m3
            o = _rows_64(*_quant_64(h)) @ _matrix_64(s["dn"][e], s["dns"][e]).t()
            out.index_add_(0, rows, o * weight[lo:hi, None])
        return out
    if c["op"] == "quant":
        q, scales = _quant_64(s["x"].double())
        return {"q": q, "s": scales}
    if c["op"] == "route":
        l = s["l"].double()
        p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
        ids = _route_plain(s)["topk"].long()      # the choice itself is whole numbers; the weights follow from it
        w = p.gather(1, ids.clamp_min(0)) * (ids >= 0)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        return {"topk": None, "weights": w * c["scale"], "seg_expert": None, "seg_offsets": None, "row_index": None,
                "slot_row": None}
    o = s["o"].double()
    if s["w1"] is not None:
        o = o / torch.sqrt(o.square().mean(1, keepdim=True) + s["eps"]) * (s["w1"].double() + c["offset"])
    if s["gate"] is not None:
        o = o * s["gate"].double().repeat_interleave(c["gate_rows"], 0)[:c["t"]]
    v = o + s["r"].double() * s["scale"]
    h = v / torch.sqrt(v.square().mean(1, keepdim=True) + s["eps"]) * (s["w2"].double() + c["offset"])
    got = {"v": v}
    if c["out"] != "fp8":
        got["h"] = h
    if c["out"] != "bf16":
        got["q"], got["s"] = _quant_64(h)
    return got
