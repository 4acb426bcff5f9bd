"""Cases of the router and microscaled 4-bit operators, their plain forms and their 64-bit results.

Three operators: routing of tokens to experts from router logits ("route"), quantisation of rows to
microscaled 4-bit floating point and back ("quantize"), and the product of activations with 4-bit
weight matrices, one per expert or a single one ("product": the activations are quantised and
multiplied, the two calls a linear layer makes).
"""
import math

import torch

own = False

# Formats: values per block scale.  "mx": blocks of 32 with a power-of-two scale; "nv": blocks of
# 16 with an e4m3 scale and one float32 power of two per row.
BLOCK = {"mx": 32, "nv": 16}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoded token through a 256-expert router with a balance bias, 4 of 8 groups kept
        _route("route_token", 1, 256, 8, 8, 4, "sigmoid", "top2", True, True, 2.5, "f32"),
        # a decode batch through a 64-expert softmax router, weights renormalised
        _route("route_batch", 32, 64, 8, 1, 1, "softmax", "max", False, True, 1.0, "bf16"),
        # a prefill step of the 256-expert layer, softmax scores, groups by their best expert
        _route("route_prefill", 2048, 256, 8, 8, 4, "softmax", "max", False, False, 2.5, "f32"),
        # a large prefill batch with a balance bias and top-2 group sums
        _route("route_large", 16384, 256, 8, 8, 4, "sigmoid", "top2", True, True, 2.5, "f32"),
        # the activations of one token
        _quantize("quantize_token", "nv", 1, 6144, "bf16", 1),
        # a prefill step's activations gathered into the slots of 8 experts per token
        _quantize("quantize_slots", "nv", 2048, 6144, "bf16", 8),
        # a weight matrix (or float32 activations) of odd height, read back after quantisation
        _quantize("quantize_rows", "mx", 5003, 2048, "f32", 1),
        # the smallest layer: 8 tokens, hidden 256, gate and up of 128 rows each
        _product("linear_tiny", "mx", 8, 1, 1, 256, 256, 0.0, "f32"),
        # one token, the 8 experts it is routed to out of 64 (gate and up rows)
        _product("experts_token", "nv", 1, 64, 8, 4096, 6144, 0.0, "bf16"),
        # a decode batch over 64 small experts, the down projection's orientation
        _product("experts_batch", "mx", 32, 64, 8, 2048, 1024, 0.0, "f32"),
        # a prefill step of a 64-expert layer with popular and rare experts
        _product("experts_prefill", "nv", 512, 64, 8, 4096, 6144, 1.1, "bf16"),
        # the shared expert's gate and up rows over a long prefill: bound by the products
        _product("linear_prefill", "nv", 8192, 1, 1, 4096, 6144, 0.0, "bf16"),
    ]


def _route(name, tokens, experts, top_k, groups, kept, score, group_score, bias, renorm, scaling, dtype):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "groups": groups, "kept": kept,
            "score": score, "group_score": group_score, "bias": bias, "renorm": renorm, "scaling": scaling, "dtype": dtype}


def _quantize(name, fmt, tokens, k, dtype, copies):
    return {"name": name, "op": "quantize", "fmt": fmt, "tokens": tokens, "k": k, "dtype": dtype, "copies": copies}


def _product(name, fmt, tokens, experts, top_k, n, k, skew, out):
    return {"name": name, "op": "product", "fmt": fmt, "tokens": tokens, "experts": experts, "top_k": top_k, "n": n, "k": k,
            "skew": skew, "out": out}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "product", "product"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 4, 1024 // groups)
        kept = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, kept * (experts // groups)))
        score = rng.choice(["softmax", "sigmoid"])
        c = _route(None, _log(rng, 1, 16384 * 256 // max(256, experts)), experts, top_k, groups, kept, score,
                   rng.choice(["max", "top2"]), rng.random() < 0.5, rng.random() < 0.5, rng.choice([1.0, 2.5]),
                   rng.choice(["f32", "bf16"]))
    elif op == "quantize":
        k = 32 * _log(rng, 1, 256)
        copies = rng.choice([1, 1, 2, 8])
        c = _quantize(None, rng.choice(["mx", "nv"]), _log(rng, 1, max(1, min(16384, 2048 * 6144 // k) // copies)), k,
                      rng.choice(["f32", "bf16"]), copies)
    else:
        fmt, out = rng.choice(["mx", "nv"]), rng.choice(["f32", "bf16"])
        if rng.random() < 0.4:
            n, k = _log(rng, 64, 6144), 32 * _log(rng, 4, 192)
            c = _product(None, fmt, _log(rng, 1, 4096), 1, 1, n, k, 0.0, out)
        else:
            experts, n, k = _log(rng, 4, 64), _log(rng, 64, 4096), 32 * _log(rng, 4, 192)
            top_k = rng.randint(1, min(8, experts))
            c = _product(None, fmt, _log(rng, 1, 512), experts, top_k, n, k, rng.choice([0.0, 1.1]), out)
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        return {"bytes": t * e * (4 if c["dtype"] == "f32" else 2) + (4 * e if c["bias"] else 0) + 8 * t * k, "flops": 0}
    if c["op"] == "quantize":
        rows, item = c["tokens"] * c["copies"], 4 if c["dtype"] == "f32" else 2
        # the source once, codes and scales once written, the values they stand for written in the source's type
        return {"bytes": c["tokens"] * c["k"] * item + rows * (c["k"] // 2 + c["k"] // BLOCK[c["fmt"]]) + rows * c["k"] * item, "flops": 0}
    rows = c["tokens"] * c["top_k"]
    used = min(c["experts"], rows)  # the matrices that this many rows reach at most
    packed = c["k"] // 2 + c["k"] // BLOCK[c["fmt"]]
    return {"bytes": c["tokens"] * c["k"] * 2 + used * c["n"] * packed + rows * c["n"] * (4 if c["out"] == "f32" else 2),
            "flops": 2 * rows * c["n"] * c["k"]}


# ------------------------------------------------------------------ inputs


def _pow2(e):
    """2**e in float32 for whole e of -126..127, from the bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _floor_log2(a):
    """floor(log2(a)) of positive float32 values."""
    return torch.frexp(a)[1] - 1


def _codes(y):
    """The e2m1 code (0..7) of magnitudes y: round to nearest, ties to the even code, saturating."""
    return ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)).to(torch.uint8)


def _quantise(x, fmt):
    """Rows of x as codes (0..15, [rows][k]), block scales (their bytes, [rows][k/block]) and row scales."""
    x = x.to(torch.float32)
    rows, k = x.shape
    b = x.view(rows, k // BLOCK[fmt], BLOCK[fmt])
    amax = b.abs().amax(2)
    if fmt == "mx":
        e = torch.where(amax > 0, _floor_log2(amax) - 2, -127).clamp(min=-127)
        scale8 = (e + 127).to(torch.uint8)
        y = b * _pow2(-e)[:, :, None]
        row = torch.ones(rows, dtype=torch.float32, device=x.device)
    else:
        top = amax.amax(1)
        e = torch.where(top > 0, _floor_log2(top) - 10, 0).clamp(min=-126)
        row, inv = _pow2(e), _pow2(-e)
        # divided by a tensor: torch multiplies by the rounded reciprocal of a number instead
        s = (amax * inv[:, None] / inv.new_full((1,), 6.0)).to(torch.float8_e4m3fn)
        scale8 = s.view(torch.uint8)
        s = s.to(torch.float32)[:, :, None]
        y = torch.where(s > 0, b * inv[:, None, None] / torch.where(s > 0, s, 1), 0)
    code = _codes(y.abs()) | (torch.signbit(y).to(torch.uint8) << 3)
    return code.view(rows, k), scale8, row


def _values(code, scale8, row, fmt):
    """The float32 values that codes, block scales and row scales stand for."""
    rows, k = code.shape
    mag = torch.tensor(E2M1, device=code.device)[(code & 7).long()]
    v = torch.where(code > 7, -mag, mag).view(rows, k // BLOCK[fmt], BLOCK[fmt])
    s = torch.where(scale8 > 0, _pow2(scale8.to(torch.int32) - 127), 2.0 ** -127) if fmt == "mx" else scale8.view(torch.float8_e4m3fn).to(torch.float32)
    return (v * s[:, :, None]).view(rows, k) * row[:, None]


def _pitch(fmt, k):
    """Bytes of a row of block scales: whole k-blocks of 256 values."""
    return (k + 255) // 256 * (256 // BLOCK[fmt])


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _tiles(scale8, fmt, k):
    """Block scales of a matrix [n][k/block] in tiles of 128 rows x 4 scales: byte (r % 32) * 16 + (r // 32) * 4 + j of a tile."""
    n, p = scale8.shape[0], _pitch(fmt, k)
    full = torch.zeros((n + 127) // 128 * 128, p, dtype=torch.uint8, device=scale8.device)
    full[:n, :scale8.shape[1]] = scale8
    return full.view(-1, 4, 32, p // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    if c["op"] == "route":
        logits = normal(c["tokens"], c["experts"]).to(DTYPE[c["dtype"]])
        bias = normal(c["experts"]) * 0.1 if c["bias"] else None
        return {"case": c, "logits": logits, "bias": bias,
                "ids": torch.empty(c["tokens"], c["top_k"], dtype=torch.int32, device="cuda"),
                "weights": torch.empty(c["tokens"], c["top_k"], device="cuda")}

    t, k, fmt = c["tokens"], c["k"], c["fmt"]
    pitch = _pitch(fmt, k)
    # a few channels are far larger than the rest, as a trained model's activations have them
    x = normal(t, k) * torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    state = {"case": c, "ws": torch.zeros(4096, dtype=torch.uint8, device="cuda")}
    if c["op"] == "quantize":
        rows = t * c["copies"]
        state["x"] = x.to(DTYPE[c["dtype"]])
        # slot -> copy of a token, in the order of the experts that the slots belong to
        state["perm"] = torch.randperm(rows, generator=g, device="cuda").to(torch.int32) if c["copies"] > 1 else None
        state["out"] = torch.empty(rows, k, dtype=DTYPE[c["dtype"]], device="cuda")
    else:
        rows, e, n = t * c["top_k"], c["experts"], c["n"]
        state["x"] = x.to(torch.bfloat16)
        state["perm"], state["offsets"], state["fullest"] = None, None, t
        if e > 1:
            # popularity of the experts: all alike, or falling with their rank
            rank = torch.randperm(e, generator=g, device="cuda").to(torch.float32) + 1
            noise = torch.rand(t, e, generator=g, device="cuda").clamp_min(1e-20).log().neg().log().neg()
            ids = (noise - 0.5 * c["skew"] * rank.log()).topk(c["top_k"], dim=1).indices.reshape(-1)
            state["perm"] = torch.sort(ids, stable=True).indices.to(torch.int32)
            counts = torch.bincount(ids, minlength=e)
            state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            state["fullest"] = int(counts.max())
        w = {"codes": torch.empty(e, n, k // 2, dtype=torch.uint8, device="cuda"),
             "tiles": torch.empty(e, (n + 127) // 128 * 128 * pitch, dtype=torch.uint8, device="cuda"),
             "row": torch.empty(e, n, device="cuda")}
        for i in range(e):
            code, s8, row = _quantise(normal(n, k) * 0.02, fmt)
            w["codes"][i], w["tiles"][i], w["row"][i] = _pack(code), _tiles(s8, fmt, k), row
        state["w"] = w
        state["out"] = torch.empty(rows, n, dtype=DTYPE[c["out"]], device="cuda")
    state["codes"] = torch.empty(rows, k // 2, dtype=torch.uint8, device="cuda")
    state["scales"] = torch.empty(rows, pitch, dtype=torch.uint8, device="cuda")
    state["row"] = torch.empty(rows, device="cuda")
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _run_route, "quantize": _run_quantize, "product": _run_product}[op](state)
    return {"route": _plain_route, "quantize": _plain_quantize, "product": _plain_product}[op](state)


def _run_route(s):
    import quantized_routed_expert_noaux_b200 as q
    c = s["case"]
    router = q.MoERouter(c["experts"], c["top_k"], c["groups"], c["kept"],
                         q.COLI_SCORE_SOFTMAX if c["score"] == "softmax" else q.COLI_SCORE_SIGMOID,
                         q.COLI_GROUP_MAX if c["group_score"] == "max" else q.COLI_GROUP_TOP2,
                         int(c["renorm"]), q.COLI_ACT_F32 if c["dtype"] == "f32" else q.COLI_ACT_BF16, c["scaling"])
    q.coli_moe_route_scores(router, s["logits"], s["logits"].stride(0), s["bias"], c["tokens"], s["ids"], s["weights"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _call_quantize(q, s, act):
    c = s["case"]
    fmt = q.COLI_FP4_MX if c["fmt"] == "mx" else q.COLI_FP4_NV
    rows = s["codes"].shape[0]
    q.coli_moe_fp4_quantize(fmt, q.COLI_FP4_ROWS, act, s["x"], s["x"].shape[0], c["k"], s["perm"], rows // s["x"].shape[0], rows, c["k"],
                            s["codes"], s["scales"], s["row"], s["ws"])
    return fmt


def _run_quantize(s):
    import quantized_routed_expert_noaux_b200 as q
    c = s["case"]
    act = q.COLI_ACT_F32 if c["dtype"] == "f32" else q.COLI_ACT_BF16
    fmt = _call_quantize(q, s, act)
    q.coli_moe_fp4_dequantize(fmt, q.COLI_FP4_ROWS, s["codes"], s["scales"], s["row"], s["codes"].shape[0], c["k"], act, s["out"], c["k"])
    return s["out"]


def _run_product(s):
    import quantized_routed_expert_noaux_b200 as q
    c, w = s["case"], s["w"]
    fmt = _call_quantize(q, s, q.COLI_ACT_BF16)
    a = q.fp4_rows_for(s["codes"], s["scales"], s["row"])
    b = q.fp4_mats_for(w["codes"], w["tiles"], w["row"])
    q.coli_moe_fp4_product(fmt, a, b, c["k"], s["offsets"], q.COLI_ACT_F32 if c["out"] == "f32" else q.COLI_ACT_BF16, s["out"], c["n"], s["ws"])
    return s["out"]


def _plain_route(s):
    c = s["case"]
    t, e = s["logits"].shape
    # in 64 bits: which expert comes first is decided by the last bits
    l = s["logits"].double()
    p = torch.exp(l - l.amax(1, keepdim=True))
    score = p / p.sum(1, keepdim=True) if c["score"] == "softmax" else 1 / (1 + torch.exp(-l))
    key = l if s["bias"] is None else score + s["bias"].double()
    if c["kept"] < c["groups"]:
        by = (score if s["bias"] is None else key).view(t, c["groups"], -1)
        best = (key.view(t, c["groups"], -1).amax(2) if c["group_score"] == "max" or by.shape[2] == 1
                else torch.sort(by, dim=2, descending=True).values[:, :, :2].sum(2))
        keep = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        dropped = torch.ones(t, c["groups"], dtype=torch.bool, device=l.device).scatter_(1, keep, False)
        key = key.masked_fill(dropped.repeat_interleave(e // c["groups"], 1), -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * c["scaling"]).to(torch.float32)}


def _source(s):
    """The rows to quantise: the tokens, or every slot's token."""
    copies = s["codes"].shape[0] // s["x"].shape[0]
    return s["x"] if s["perm"] is None else s["x"][torch.div(s["perm"].long(), copies, rounding_mode="floor")]


def _plain_quantize(s):
    fmt = s["case"]["fmt"]
    return _values(*_quantise(_source(s), fmt), fmt).to(s["x"].dtype)


def _weights(w, fmt, k):
    """The float32 matrices [experts][n][k] that packed codes, tiled block scales and row scales stand for."""
    e, n, _ = w["codes"].shape
    code = torch.stack([w["codes"] & 15, w["codes"] >> 4], 3).view(e * n, k)
    s8 = w["tiles"].view(e, (n + 127) // 128, -1, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(e, (n + 127) // 128 * 128, -1)
    return _values(code, s8[:, :n, :k // BLOCK[fmt]].reshape(e * n, -1), w["row"].view(-1), fmt).view(e, n, k)


def _plain_product(s):
    c = s["case"]
    x = _values(*_quantise(_source(s), c["fmt"]), c["fmt"])
    w = _weights(s["w"], c["fmt"], c["k"])
    if s["offsets"] is None:
        return torch.matmul(x, w[0].t()).to(s["out"].dtype)
    # every expert's rows side by side in one batch, as many as the fullest one has
    off = s["offsets"].long()
    at = torch.arange(x.shape[0], device=x.device)
    expert = torch.searchsorted(off[1:], at, right=True)
    place = at - off[expert]
    batch = torch.zeros(c["experts"], s["fullest"], c["k"], device=x.device)
    batch[expert, place] = x
    return torch.bmm(batch, w.transpose(1, 2))[expert, place].to(s["out"].dtype)


# ------------------------------------------------------------------ 64-bit results


def _exact_pow2(e):
    """2**e in float64 for whole e, from the bits (pow is not exact on the GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_log2(a):
    """floor(log2(a)) of positive values, 0 for zero."""
    return torch.frexp(torch.where(a > 0, a, 1.0)).exponent.long() - 1


def _exact_rounded(v, mantissa, lowest, most):
    """v (float64, >= 0) rounded to `mantissa` fraction bits with lowest exponent `lowest`, ties to even, at most `most`."""
    step = _exact_pow2(_exact_log2(v).clamp(min=lowest) - mantissa)
    return torch.clamp(torch.round(v / step) * step, max=most)


def _exact_quantised(x, fmt):
    """The float64 values that rows of x become."""
    v = x.double()
    rows, k = v.shape
    b = v.reshape(rows, -1, BLOCK[fmt])
    amax = b.abs().max(2, keepdim=True).values
    if fmt == "mx":
        scale = _exact_pow2(torch.where(amax > 0, _exact_log2(amax) - 2, -127).clamp(min=-127))
    else:
        top = amax.max(1, keepdim=True).values
        r = _exact_pow2(torch.where(top > 0, _exact_log2(top) - 10, 0).clamp(min=-126))
        scale = _exact_rounded(amax / (6 * r), 3, -6, 448.0) * r
    y = torch.where(scale > 0, b.abs() / torch.where(scale > 0, scale, 1.0), 0.0)
    return (torch.sign(b) * _exact_rounded(y, 1, 0, 6.0) * scale).reshape(rows, k)


def _exact_weights(w, fmt, k, i):
    """Matrix i in float64, from its bytes."""
    packed = w["codes"][i].long()
    n = packed.shape[0]
    code = torch.empty(n, k, dtype=torch.long, device=packed.device)
    code[:, 0::2], code[:, 1::2] = packed % 16, packed // 16
    mantissa, exponent = (code % 2).double(), code // 2 % 4
    v = torch.where(exponent > 0, (1 + mantissa / 2) * _exact_pow2(exponent - 1), mantissa / 2) * torch.where(code > 7, -1.0, 1.0)
    r = torch.arange(n, device=packed.device)[:, None]
    j = torch.arange(k // BLOCK[fmt], device=packed.device)[None, :]
    at = (r // 128) * (_pitch(fmt, k) * 128) + (j // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + j % 4
    byte = w["tiles"][i].long()[at]
    if fmt == "mx":
        s = _exact_pow2(byte - 127)
    else:
        m, e = (byte % 8).double(), byte // 8
        s = torch.where(e > 0, (1 + m / 8) * _exact_pow2(e - 7), m / 8 * 2.0 ** -6)
    return v * s.repeat_interleave(BLOCK[fmt], 1) * w["row"][i].double()[:, None]


def _exact_route(s):
    c = s["case"]
    logit = s["logits"].to(torch.float64)
    t, e = logit.shape
    if c["score"] == "softmax":
        score = torch.exp(logit - torch.logsumexp(logit, 1, keepdim=True))
    else:
        score = torch.sigmoid(logit)
    value = logit if s["bias"] is None else score + s["bias"].double()
    size = e // c["groups"]
    if c["kept"] < c["groups"]:
        sums = score if s["bias"] is None else value
        if c["group_score"] == "max" or size == 1:
            best = value.reshape(t, -1, size).max(2).values
        else:
            best = sums.reshape(t, -1, size).topk(2, 2).values.sum(2)
        # a group's place: how many come before it (a larger value, or the same and a lower index)
        before = (best[:, None, :] > best[:, :, None]).sum(2)
        lower = torch.tril(torch.ones(c["groups"], c["groups"], dtype=torch.bool, device=best.device), -1)
        before = before + ((best[:, None, :] == best[:, :, None]) & lower).sum(2)
        value = torch.where((before < c["kept"]).repeat_interleave(size, 1), value, -math.inf)
    ids = torch.argsort(-value, dim=1, stable=True)[:, :c["top_k"]]
    w = torch.gather(score, 1, ids)
    w = w / (w.sum(1, keepdim=True) if c["renorm"] else 1.0) * c["scaling"]
    return {"ids": None, "weights": w}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "route":
        return _exact_route(s)
    x = s["x"]
    if s["perm"] is not None:
        x = x.index_select(0, s["perm"].long() // (s["codes"].shape[0] // x.shape[0]))
    v = _exact_quantised(x, c["fmt"])
    if c["op"] == "quantize":
        return v
    if s["offsets"] is None:
        return v @ _exact_weights(s["w"], c["fmt"], c["k"], 0).t()
    ends = s["offsets"].tolist()
    parts = [v[ends[i]:ends[i + 1]] @ _exact_weights(s["w"], c["fmt"], c["k"], i).t() for i in range(c["experts"]) if ends[i + 1] > ends[i]]
    return torch.cat(parts)
