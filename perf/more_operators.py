"""Cases that measure the products of two microscaled 4-bit operands and the mixture-of-experts
layer for a few tokens, both on packed MXFP4 weights.

``own = False`` computes each operator in its plain form with elementary torch operations in
32 bits; ``own = True`` makes the library's calls.  Both take the same state from ``prepare``:
inputs, and weights in the canonical layout of ``include/qmm.h`` as well as packed once.

Formulas (b: blocks of 32 along the reduction axis)
  quant    m = max_b |x|;  E = floor(log2 m) - 2 + 127 ("floor"), or the smallest E with
           m <= 6 * 2^(E-127) ("fit"), held to 0 .. 254;  q = E2M1(x * 2^(127-E)), nearest, ties
           to even, at most 6.  Scaling by a power of two is exact: codes follow from x alone
  linear   x quantised, then y[t,n] = sum_b 2^(Ex[t,b]-127) * 2^(Ew[n,b]-127) * sum_{k in b} q[t,k] * w[n,k]
  experts  per routed row: h = silu(x G^T) * (x U^T) on quantised x, h quantised from its 32-bit
           value, times the down matrix; out[t] = sum_j weight[t,j] * o[row of slot j]
  moe      s = softmax(l) or sigmoid(l); the k best experts (of the best groups, by s + bias);
           out[t] = sum_j weight[t,j] * D_e (silu(G_e x) * (U_e x)) (+ shared[t]), x and weights' products not quantised
"""
import math
import struct

import torch

own = False

DEV = "cuda"
BLOCK = 32
SLAB = 512                 # codes of one slab of the packed layout
MXFP4 = 2                  # the library's code of the weight format
RULES = {"floor": 0, "fit": 1}
BF16, F32 = 1, 2           # the library's type codes
SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode token against a wide projection: the weights' bytes are the whole cost
        {"name": "linear_decode", "op": "linear", "t": 1, "n": 13824, "d": 5120, "rule": "fit"},
        # an odd decode batch on the narrower way back
        {"name": "linear_batch", "op": "linear", "t": 47, "n": 5120, "d": 13824, "rule": "fit"},
        # a short ragged prompt: no size is a multiple of a tile, the last slab is short
        {"name": "linear_ragged", "op": "linear", "t": 333, "n": 1000, "d": 2080, "rule": "floor"},
        # prefill of one sequence: the matrix cores' rate
        {"name": "linear_prefill", "op": "linear", "t": 2048, "n": 13824, "d": 5120, "rule": "fit"},
        # a long prefill of a square projection
        {"name": "linear_long", "op": "linear", "t": 8192, "n": 8192, "d": 8192, "rule": "floor"},
        # a decode batch through routed experts: about four rows an expert
        {"name": "experts_batch", "op": "experts", "t": 64, "experts": 128, "k": 8, "d": 3584, "inter": 2048, "rule": "fit"},
        # a routed prompt of odd sizes
        {"name": "experts_ragged", "op": "experts", "t": 517, "experts": 60, "k": 4, "d": 2080, "inter": 1056, "rule": "floor"},
        # routed prefill: hundreds of rows an expert
        {"name": "experts_prefill", "op": "experts", "t": 4096, "experts": 64, "k": 8, "d": 3584, "inter": 2048, "rule": "fit"},
        # one decode token, sigmoid scores with a balance bias and expert groups
        {"name": "moe_one", "op": "moe", "t": 1, "experts": 256, "k": 8, "d": 3584, "inter": 2048, "score": "sigmoid",
         "bias": True, "groups": 8, "keep": 4, "by": "top2", "renorm": True, "scale": 2.5, "logits": "f32", "shared": True},
        # the smallest layer: latency
        {"name": "moe_small", "op": "moe", "t": 2, "experts": 8, "k": 2, "d": 1024, "inter": 512, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "by": "max", "renorm": True, "scale": 1.0, "logits": "f32", "shared": False},
        # a few sequences, odd sizes, bf16 logits (exact ties)
        {"name": "moe_odd", "op": "moe", "t": 7, "experts": 60, "k": 4, "d": 2080, "inter": 1056, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "by": "max", "renorm": False, "scale": 1.0, "logits": "bf16", "shared": True},
        # the largest decode batch of the layer: nearly every expert has a row
        {"name": "moe_sixteen", "op": "moe", "t": 16, "experts": 64, "k": 8, "d": 3584, "inter": 2048, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "by": "max", "renorm": True, "scale": 1.0, "logits": "bf16", "shared": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "experts", "moe", "moe"])
    if op == "linear":
        while True:
            c = {"op": op, "t": _log(rng, 1, 8192), "n": _log(rng, 64, 14336), "d": 32 * _log(rng, 4, 512),
                 "rule": rng.choice(["floor", "fit"])}
            if c["t"] * c["n"] * c["d"] <= 8192 ** 3 and c["n"] * c["d"] >= 1 << 17:
                return c
    if op == "experts":
        while True:
            c = {"op": op, "t": _log(rng, 1, 4096), "experts": rng.choice([8, 16, 60, 64, 128]), "k": rng.randint(1, 8),
                 "d": 32 * _log(rng, 16, 128), "inter": 32 * _log(rng, 8, 64), "rule": rng.choice(["floor", "fit"])}
            if (c["t"] * c["k"] * c["d"] * c["inter"] <= 4096 * 8 * 3584 * 2048
                    and c["experts"] * c["d"] * c["inter"] <= 64 * 3584 * 2048):
                return c
    while True:
        experts, groups = rng.choice([(8, 1), (16, 1), (60, 1), (64, 8), (128, 1), (160, 8), (256, 8), (384, 1)])
        score = rng.choice(["softmax", "sigmoid"])
        c = {"op": op, "t": rng.randint(1, 16), "experts": experts, "k": rng.randint(1, 8), "d": 32 * _log(rng, 16, 224),
             "inter": 32 * _log(rng, 8, 96), "score": score, "bias": score == "sigmoid" and rng.random() < 0.7,
             "groups": groups, "keep": max(1, groups // 2), "by": "max" if score == "softmax" else rng.choice(["max", "top2"]),
             "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "logits": rng.choice(["f32", "bf16"]),
             "shared": rng.random() < 0.5}
        if (c["experts"] * c["d"] * c["inter"] <= 256 * 3584 * 2048
                and c["t"] * c["k"] * c["d"] * c["inter"] <= 16 * 8 * 3584 * 2048):
            return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFFFFFF)


def _activations(g, t, d):
    """bf16 rows as a norm leaves them: near normal, a few channels much larger."""
    x = torch.randn(t, d, generator=g, device=DEV)
    wide = (torch.rand(d, generator=g, device=DEV) < 0.004).float() * 12.0 + 1.0
    return (x * wide).to(torch.bfloat16)


def _canonical(w):
    """Codes uint8[n][d/2] and E8M0 uint8[n][d/32] of a matrix, by the rule "fit"."""
    v, e = _codes_plain(w, "fit")
    a = v.abs()
    code = torch.where(a < 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)).to(torch.uint8)
    code |= (v < 0.0).to(torch.uint8) << 3
    return code[:, 0::2] | code[:, 1::2] << 4, e.to(torch.uint8)


def _packed(codes, e8m0):
    """The packed blob of one matrix: a header of 256 bytes, the codes slab by slab (512 codes of
    every row), the exponents by fours of rows, a slab of each row padded to 4 bytes."""
    n, d = codes.shape[0], 2 * codes.shape[1]
    parts = [codes[:, s:s + SLAB // 2].reshape(-1) for s in range(0, d // 2, SLAB // 2)]
    body = torch.cat(parts)
    four = torch.nn.functional.pad(e8m0, (0, 0, 0, -n % 4))
    meta = []
    for s in range(0, d // BLOCK, SLAB // BLOCK):
        part = four[:, s:s + SLAB // BLOCK]
        meta.append(torch.nn.functional.pad(part, (0, -part.shape[1] % 4)).reshape(four.shape[0] // 4, -1))
    meta = torch.cat(meta, 1).reshape(-1)
    at = -(-(256 + n * d // 2) // 256) * 256
    total = -(-(at + meta.numel()) // 256) * 256
    head = struct.pack("<IIIIqqqqq", 0x344D4D51, 4, MXFP4, 0, n, d, 256, at, total)
    blob = torch.zeros(total, dtype=torch.uint8, device=DEV)
    blob[:len(head)] = torch.tensor(list(head), dtype=torch.uint8, device=DEV)
    blob[256:256 + body.numel()] = body
    blob[at:at + meta.numel()] = meta
    return blob


def _matrix(g, n, d):
    w = torch.randn(n, d, generator=g, device=DEV) * (0.5 + torch.rand(n, 1, generator=g, device=DEV)) * d ** -0.5
    return _canonical(w)


def _weights(g, n, d):
    codes, e8m0 = _matrix(g, n, d)
    return codes, e8m0, _packed(codes, e8m0)


def _expert_weights(g, experts, n, d):
    """A stack of expert matrices, canonical and packed."""
    codes = torch.empty(experts, n, d // 2, dtype=torch.uint8, device=DEV)
    e8m0 = torch.empty(experts, n, d // BLOCK, dtype=torch.uint8, device=DEV)
    blobs = None
    for e in range(experts):
        codes[e], e8m0[e], blob = _weights(g, n, d)
        if blobs is None:
            blobs = torch.empty(experts, blob.numel(), dtype=torch.uint8, device=DEV)
        blobs[e] = blob
    return codes, e8m0, blobs


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


def _scale_bytes(d):
    return 16 * -(-d // SLAB)


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c}
    empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    bf, u8 = torch.bfloat16, torch.uint8
    if c["op"] == "linear":
        t, n, d = c["t"], c["n"], c["d"]
        s["x"] = _activations(g, t, d)
        s["w"], s["we"], s["packed"] = _weights(g, n, d)
        s["xq"], s["xe"] = empty(t, d // 2, dtype=u8), empty(t, _scale_bytes(d), dtype=u8)
        s["y"] = empty(t, n, dtype=bf)
        return s
    t, e, k, d, i = c["t"], c["experts"], c["k"], c["d"], c["inter"]
    s["x"] = _activations(g, t, d)
    s["gu"], s["gue"], s["gu_packed"] = _expert_weights(g, e, 2 * i, d)
    s["dn"], s["dne"], s["dn_packed"] = _expert_weights(g, e, d, i)
    s["out"] = empty(t, d, dtype=bf)
    if c["op"] == "experts":
        s |= _routing(g, t, e, k)
        s["most"] = int((s["seg_offsets"][1:] - s["seg_offsets"][:-1]).max())
        m = t * k
        s["xq"], s["xe"] = empty(t, d // 2, dtype=u8), empty(t, _scale_bytes(d), dtype=u8)
        s["hq"], s["he"] = empty(m, i // 2, dtype=u8), empty(m, _scale_bytes(i), dtype=u8)
        s["o"] = empty(m, d, dtype=bf)
        return s
    l = torch.randn(t, e, generator=g, device=DEV) * 1.5 + 0.5 * torch.randn(e, generator=g, device=DEV)
    s["l"] = l if c["logits"] == "f32" else l.to(bf)
    s["bias"] = 0.1 * torch.randn(e, generator=g, device=DEV) if c["bias"] else None
    s["shared"] = _activations(g, t, d) if c["shared"] else None
    s["topk"], s["weights"] = empty(t, k, dtype=torch.int32), empty(t, k, dtype=torch.float32)
    s["ws"] = empty(2 * t * k * i, dtype=u8)          # h of every slot in bf16
    return s


# ---------------------------------------------------------------- plain forms

def _codes_plain(x, rule):
    """(values of the codes, exponents) of rows."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    most = b.abs().amax(-1)
    up = 0x3FFFFF if rule == "fit" else 0             # carries into the exponent where the mantissa is over 1.5
    e = ((most.contiguous().view(torch.int32) + up >> 23) - 2).clamp(0, 254)
    v = b * torch.exp2((127 - e).float())[..., None]
    a = v.abs().clamp_max(6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v).flatten(-2), e


def _quant_plain(x, rule):
    """Rows as their codes stand for them."""
    v, e = _codes_plain(x, rule)
    return (v.unflatten(-1, (-1, BLOCK)) * torch.exp2((e - 127).float())[..., None]).flatten(-2)


def _dequant_plain(codes, e8m0):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    a = (c & 7).float()
    v = torch.where(a < 4.0, 0.5 * a, torch.where(a < 6.0, a - 2.0, 2.0 * a - 8.0))
    v = torch.where(c > 7, -v, v)
    return (v.unflatten(-1, (-1, BLOCK)) * torch.exp2(e8m0.float() - 127.0)[..., None]).flatten(-2)


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _experts_plain(s):
    c, most = s["case"], s["most"]
    i, m = c["inter"], c["t"] * c["k"]
    # the rows of every expert, padded to the longest segment
    at = s["seg_offsets"][:-1, None] + torch.arange(most, device=DEV)
    live = at < s["seg_offsets"][1:, None]
    at = at.clamp_max(m - 1)
    x = _quant_plain(s["x"], c["rule"])[s["row_index"][at]]
    y = torch.bmm(_dequant_plain(s["gu"], s["gue"]), x.transpose(1, 2).contiguous())
    del x
    h = _quant_plain((_silu(y[:, :i]) * y[:, i:]).transpose(1, 2), c["rule"])
    o = torch.bmm(_dequant_plain(s["dn"], s["dne"]), h.transpose(1, 2).contiguous())
    o = o.transpose(1, 2)[live].to(torch.bfloat16)          # grouped order again
    return (o[s["slot_row"]].float() * s["weights"][..., None]).sum(1).to(torch.bfloat16)


def _route_plain(s):
    """(ids, weights): the choice of a token's experts."""
    c, l = s["case"], s["l"].float()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
        rank = p
    else:
        z = torch.exp(l - l.amax(1, keepdim=True))
        p = z / z.sum(1, keepdim=True)
        rank = l                       # ranked by the logits themselves where no bias is added
    if s["bias"] is not None:
        rank = p + s["bias"]
    if c["groups"] > 1:
        two = rank.view(c["t"], c["groups"], -1).sort(-1, descending=True).values[..., :2]
        value = two[..., 0] if c["by"] == "max" else two[..., 0] + two[..., 1]
        kept = value.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
        rank = rank.masked_fill(~keep.repeat_interleave(c["experts"] // c["groups"], 1), -math.inf)
    ids = rank.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids, w * c["scale"]


def _moe_plain(s):
    c = s["case"]
    t, k, d, i = c["t"], c["k"], c["d"], c["inter"]
    ids, w = _route_plain(s)
    flat = ids.reshape(-1)
    x = s["x"].float().repeat_interleave(k, 0)[..., None]
    y = torch.bmm(_dequant_plain(s["gu"][flat], s["gue"][flat]), x)[..., 0]
    h = (_silu(y[:, :i]) * y[:, i:])[..., None]
    o = torch.bmm(_dequant_plain(s["dn"][flat], s["dne"][flat]), h).view(t, k, d)
    out = (o * w[..., None]).sum(1)
    if s["shared"] is not None:
        out = out + s["shared"].float()
    return {"topk": ids.to(torch.int32), "weights": w, "out": out.to(torch.bfloat16)}


# ---------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "linear":
            return (_quant_plain(s["x"], c["rule"]) @ _dequant_plain(s["w"], s["we"]).t()).to(torch.bfloat16)
        return _experts_plain(s) if c["op"] == "experts" else _moe_plain(s)
    import bit_weight_quantized_amd as qmm
    if c["op"] == "linear":
        t, n, d = c["t"], c["n"], c["d"]
        qmm.qmm_mxfp4_quant(s["x"], t, d, d, RULES[c["rule"]], s["xq"], s["xe"])
        qmm.qmm_mxfp4_gemm(s["packed"], t, n, d, s["xq"], s["xe"], s["y"], n)
        return s["y"]
    t, e, k, d, i = c["t"], c["experts"], c["k"], c["d"], c["inter"]
    gu, dn = s["gu_packed"], s["dn_packed"]
    if c["op"] == "experts":
        m, rule = t * k, RULES[c["rule"]]
        table = (s["seg_expert"], s["seg_offsets"], e, m, t)
        qmm.qmm_mxfp4_quant(s["x"], t, d, d, rule, s["xq"], s["xe"])
        qmm.qmm_mxfp4_grouped_gemm_swiglu(gu, gu.shape[1], e, 2 * i, d, s["xq"], s["xe"], t, s["row_index"], *table, rule,
                                          None, s["hq"], s["he"])
        qmm.qmm_mxfp4_grouped_gemm(dn, dn.shape[1], e, d, i, s["hq"], s["he"], m, None, *table, s["o"])
        qmm.qmm_moe_gather(s["o"], m, d, t, k, s["slot_row"], s["weights"], None, s["out"])
        return s["out"]
    qmm.qmm_moe_layer(MXFP4, gu, gu.shape[1], dn, dn.shape[1], e, d, i, s["x"], t, s["l"],
                      BF16 if c["logits"] == "bf16" else F32, e, SIGMOID if c["score"] == "sigmoid" else SOFTMAX, s["bias"],
                      c["groups"], c["keep"], GROUP_TOP2 if c["by"] == "top2" else GROUP_MAX, k, c["renorm"], c["scale"],
                      s["shared"], s["topk"], s["weights"], s["out"], s["ws"])
    return {"topk": s["topk"], "weights": s["weights"], "out": s["out"]}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "linear":
        t, n, d = c["t"], c["n"], c["d"]
        return {"bytes": n * d * 17 // 32 + 2 * t * d + 2 * t * n, "flops": 2 * t * n * d}
    t, e, k, d, i = c["t"], c["experts"], c["k"], c["d"], c["inter"]
    used = e * (1.0 - (1.0 - k / e) ** t)              # experts that get a row, expected
    each = int(used * 3 * i * d * 17 / 32)
    rest = 8 * t * k if c["op"] == "experts" else t * e * (4 if c["logits"] == "f32" else 2) + 8 * t * k + 2 * t * d * c["shared"]
    return {"bytes": each + 4 * t * d + rest, "flops": 6 * t * k * i * d}


# ---------------------------------------------------------------- the definitions in 64 bits

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _rows_64(x, rule):
    """Quantised rows in 64 bits: the nearest of the eight magnitudes, a midpoint to the even code."""
    table = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    middle = (table[1:] + table[:-1]) / 2
    b = x.double().reshape(*x.shape[:-1], -1, BLOCK)
    most = b.abs().max(-1, keepdim=True).values
    if rule == "floor":
        e = torch.frexp(most).exponent - 1 - 2
    else:
        mantissa, e = torch.frexp(most / 6.0)          # most / 6 in [1/2, 1) * 2^e, a power of two where the mantissa is 1/2
        e = e - (mantissa == 0.5).to(e.dtype)
    scale = torch.exp2(torch.where(most > 0, e, -127).clamp(-127, 127).double())
    a = b.abs() / scale
    low = torch.bucketize(a, middle)                   # midpoints below a
    high = torch.bucketize(a, middle, right=True)      # midpoints not above a
    code = torch.where(low % 2 == 0, low, high)        # on a midpoint they differ by one: the even one
    return (torch.copysign(table[code], b) * scale).reshape(x.shape)


def _matrix_64(codes, e8m0):
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=codes.device)
    v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    v[:, 0::2] = table[(codes & 15).long()]
    v[:, 1::2] = table[(codes >> 4).long()]
    return v * torch.exp2(e8m0.double() - 127.0).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        return _rows_64(s["x"], c["rule"]) @ _matrix_64(s["w"], s["we"]).t()
    t, k, i = c["t"], c["k"], c["inter"]
    if c["op"] == "experts":
        x, offsets = _rows_64(s["x"], c["rule"]), s["seg_offsets"].tolist()
        weight = torch.empty(t * k, dtype=torch.float64, device=DEV)
        weight[s["slot_row"].reshape(-1).long()] = s["weights"].double().reshape(-1)
        segments = [(e, s["row_index"][lo:hi].long(), weight[lo:hi]) for e, (lo, hi) in enumerate(zip(offsets, offsets[1:]))]
    else:
        x, ids = s["x"].double(), _route_plain(s)[0]   # the choice itself is whole numbers; the weights follow from it
        l = s["l"].double()
        p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
        w = p.gather(1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = w * c["scale"]
        segments = []
        for e in sorted(set(ids.reshape(-1).tolist())):
            token, slot = torch.nonzero(ids == e, as_tuple=True)
            segments.append((e, token, w[token, slot]))
    out = torch.zeros(t, c["d"], dtype=torch.float64, device=DEV)
    for e, rows, weight in segments:
        if rows.numel():
            gate_up = x[rows] @ _matrix_64(s["gu"][e], s["gue"][e]).t()
            gate, up = gate_up[:, :i], gate_up[:, i:]
            h = gate * torch.sigmoid(gate) * up
            if c["op"] == "experts":
                h = _rows_64(h, c["rule"])
            out.index_add_(0, rows, (h @ _matrix_64(s["dn"][e], s["dne"][e]).t()) * weight[:, None])
    if c["op"] == "experts":
        return out
    return {"topk": None, "weights": w, "out": out if s["shared"] is None else out + s["shared"].double()}
