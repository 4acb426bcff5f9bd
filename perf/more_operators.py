"""Cases of the operators that move tokens to their experts and back, and of the 8-bit products, with their plain
forms and their 64-bit results.

Four operators: the slots of a routed batch sorted by expert with their tokens' rows ("sort"), the weighted sum
of every token's expert rows ("combine"; without weights and addend it is the gradient of the sort), the gradient of that
sum in the rows and in the weights ("grad"), and the product of rows with 8-bit weight matrices, one per expert or a
single one ("product": rows are quantised to 8 bits with a scale each, SwiGLU applied first for a down projection, and
multiplied: the two calls a linear layer makes).
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoded token of the 256-expert layer
        _sort("sort_token", 1, 256, 8, 6144, "bf16", 0.0, 0.0),
        # a prefill step of that layer with popular and rare experts
        _sort("sort_prefill", 2048, 256, 8, 6144, "bf16", 1.1, 0.0),
        # rows of odd length, a quarter of the slots on experts that live elsewhere
        _sort("sort_ragged", 777, 64, 6, 1001, "f32", 0.0, 0.25),
        # one decoded token back, the shared expert's row added
        _combine("combine_token", 1, 8, 6144, "bf16", "f32", True, True, 0.0),
        # the prefill step back
        _combine("combine_prefill", 2048, 8, 6144, "bf16", "f32", True, True, 0.0),
        # a training step of the 64-expert layer: the gradient of its sorted rows
        _combine("sort_grad", 8192, 8, 2048, "bf16", "bf16", False, False, 0.0),
        # the gradient of the weighted sum in a small batch, rows of odd length, some slots elsewhere
        _grad("grad_batch", 61, 6, 1001, "f32", "f32", 0.25),
        # in the training step of the 64-expert layer
        _grad("grad_train", 8192, 8, 2048, "bf16", "bf16", 0.0),
        # the smallest layer: 8 tokens, hidden 256, gate and up of 128 rows each
        _product("linear_tiny", 8, 1, 1, 256, 256, False, 0.0, "f32", "f32"),
        # one token, the 8 experts it is routed to out of 64 (gate and up rows)
        _product("experts_token", 1, 64, 8, 4096, 6144, False, 0.0, "bf16", "bf16"),
        # the down projections of a prefill step with popular and rare experts
        _product("experts_down", 512, 64, 8, 6144, 2048, True, 1.1, "bf16", "bf16"),
        # the shared expert's gate and up rows over a long prefill: bound by the products
        _product("linear_prefill", 8192, 1, 1, 4096, 6144, False, 0.0, "bf16", "bf16"),
    ]


def _sort(name, tokens, experts, top_k, hidden, dtype, skew, masked):
    return {"name": name, "op": "sort", "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden, "dtype": dtype,
            "skew": skew, "masked": masked}


def _combine(name, tokens, top_k, hidden, dtype, out, weights, add, masked):
    return {"name": name, "op": "combine", "tokens": tokens, "top_k": top_k, "hidden": hidden, "dtype": dtype, "out": out,
            "weights": weights, "add": add, "masked": masked}


def _grad(name, tokens, top_k, hidden, dtype, out, masked):
    return {"name": name, "op": "grad", "tokens": tokens, "top_k": top_k, "hidden": hidden, "dtype": dtype, "out": out, "masked": masked}


def _product(name, tokens, experts, top_k, n, k, glu, skew, dtype, out):
    return {"name": name, "op": "product", "tokens": tokens, "experts": experts, "top_k": top_k, "n": n, "k": k, "glu": glu,
            "skew": skew, "dtype": dtype, "out": out}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "combine", "grad", "product", "product"])
    dtype, out = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    masked = rng.choice([0.0, 0.0, 0.25])
    if op == "product":
        if rng.random() < 0.4:
            tokens, experts, top_k, n, k = _log(rng, 1, 4096), 1, 1, _log(rng, 64, 6144), _log(rng, 64, 6144)
        else:
            tokens, experts, n, k = _log(rng, 1, 512), _log(rng, 4, 64), _log(rng, 64, 4096), _log(rng, 64, 6144)
            top_k = rng.randint(1, min(8, experts))
        glu = rng.random() < 0.3
        # the rows of a down projection go to the combine in bf16
        c = _product(None, tokens, experts, top_k, n, k, glu, rng.choice([0.0, 1.1]), "bf16" if glu else dtype, "bf16" if glu else out)
    else:
        experts = _log(rng, 4, 512)
        top_k = rng.randint(1, min(16, experts))
        hidden = _log(rng, 33, 8192)
        tokens = _log(rng, 1, max(2, min(16384, 2048 * 8 * 6144 // (top_k * hidden * (2 if dtype == "f32" else 1)))))
        if op == "sort":
            c = _sort(None, tokens, experts, top_k, hidden, dtype, rng.choice([0.0, 1.1]), masked)
        elif op == "combine":
            c = _combine(None, tokens, top_k, hidden, dtype, out, rng.random() < 0.7, rng.random() < 0.5, masked)
        else:
            c = _grad(None, tokens, top_k, hidden, dtype, out, masked)
    del c["name"]
    return c


def _item(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    c = case
    if c["op"] == "product":
        rows = c["tokens"] * c["top_k"]
        used = min(c["experts"], rows)  # the matrices that this many rows reach at most
        source = rows * 2 * c["k"] if c["glu"] else c["tokens"] * c["k"]
        return {"bytes": source * _item(c["dtype"]) + used * c["n"] * (c["k"] + 4) + rows * c["n"] * _item(c["out"]),
                "flops": 2 * rows * c["n"] * c["k"]}
    t, slots, h = c["tokens"], c["tokens"] * c["top_k"], c["hidden"]
    live = int(slots * (1 - c["masked"]))
    if c["op"] == "sort":
        return {"bytes": t * h * _item(c["dtype"]) + live * h * _item(c["dtype"]) + 12 * slots + 4 * (c["experts"] + 1), "flops": 0}
    if c["op"] == "combine":
        return {"bytes": live * h * _item(c["dtype"]) + t * h * _item(c["out"]) * (2 if c["add"] else 1) + slots * (8 if c["weights"] else 4),
                "flops": 2 * live * h}
    return {"bytes": 2 * live * h * _item(c["dtype"]) + t * h * _item(c["out"]) + 12 * slots, "flops": 3 * live * h}


# ------------------------------------------------------------------ inputs


def _experts(c, g):
    """Expert ids [tokens][top_k], all different within a token: popularity alike, or falling with the experts' rank."""
    t, e = c["tokens"], c["experts"]
    rank = torch.randperm(e, generator=g, device="cuda").to(torch.float32) + 1
    noise = torch.rand(t, e, generator=g, device="cuda").clamp_min(1e-20).log().neg().log().neg()
    return (noise - 0.5 * c["skew"] * rank.log()).topk(c["top_k"], dim=1).indices


def _places(c, g):
    """Row of every slot in a grouped order [tokens][top_k] (-1: the slot is elsewhere)."""
    n = c["tokens"] * c["top_k"]
    dead = torch.rand(n, generator=g, device="cuda") < c["masked"]
    key = torch.rand(n, generator=g, device="cuda") + dead  # the rows that have none come last
    place = torch.argsort(torch.argsort(key))
    return torch.where(dead, -1, place).to(torch.int32).view(c["tokens"], c["top_k"])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def weights(t, k):  # routing weights: positive, of sum 1 to a token
        w = torch.rand(t, k, generator=g, device="cuda") + 0.05
        return w / w.sum(1, keepdim=True)

    state = {"case": c, "ws": torch.zeros(4096, dtype=torch.uint8, device="cuda")}
    t = c["tokens"]
    if c["op"] == "product":
        return _prepare_product(c, g, normal, state)
    slots, h, act = t * c["top_k"], c["hidden"], DTYPE[c["dtype"]]
    if c["op"] == "sort":
        ids = _experts(c, g).to(torch.int32)
        if c["masked"]:
            ids = torch.where(torch.rand(t, c["top_k"], generator=g, device="cuda") < c["masked"], -1, ids)
        state.update(x=normal(t, h).to(act), ids=ids, rows=torch.zeros(slots, h, dtype=act, device="cuda"),
                     offsets=torch.empty(c["experts"] + 1, dtype=torch.int32, device="cuda"),
                     perm=torch.empty(slots, dtype=torch.int32, device="cuda"), place=torch.empty(slots, dtype=torch.int32, device="cuda"))
        return state
    out = DTYPE[c["out"]]
    state.update(y=normal(slots, h).to(act), place=_places(c, g))
    if c["op"] == "combine":
        state.update(w=weights(t, c["top_k"]) if c["weights"] else None, add=normal(t, h).to(out) if c["add"] else None,
                     out=torch.empty(t, h, dtype=out, device="cuda"))
    else:
        state.update(w=weights(t, c["top_k"]), dout=normal(t, h).to(out), dy=torch.zeros(slots, h, dtype=act, device="cuda"),
                     dw=torch.empty(t, c["top_k"], device="cuda"))
    return state


def _prepare_product(c, g, normal, state):
    t, k, e, n = c["tokens"], c["k"], c["experts"], c["n"]
    rows, pitch = t * c["top_k"], (k + 15) // 16 * 16
    state.update(place=None, offsets=None, fullest=t)
    if e > 1:
        ids = _experts(c, g).reshape(-1)
        perm = torch.sort(ids, stable=True).indices
        counts = torch.bincount(ids, minlength=e)
        state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        state["fullest"] = int(counts.max())
        if not c["glu"]:  # (the rows of a down projection are in their order already)
            state["place"] = torch.argsort(perm).to(torch.int32)
    # a few channels are far larger than the rest, as a trained model's activations have them
    loud = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    x = torch.cat([normal(rows, k) * 2, normal(rows, k) * loud], 1) if c["glu"] else normal(t, k) * loud
    codes = torch.zeros(e, n, pitch, dtype=torch.int8, device="cuda")
    codes[:, :, :k] = torch.randint(-127, 128, (e, n, k), generator=g, device="cuda", dtype=torch.int8)
    state.update(x=x.to(DTYPE[c["dtype"]]), wc=codes, wscale=(torch.rand(e, n, generator=g, device="cuda") + 0.5) * 3e-4,
                 codes=torch.empty(rows, pitch, dtype=torch.int8, device="cuda"), scale=torch.empty(rows, device="cuda"),
                 out=torch.empty(rows, n, dtype=DTYPE[c["out"]], device="cuda"))
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"sort": _run_sort, "combine": _run_combine, "grad": _run_grad, "product": _run_product}[op](state)
    return {"sort": _plain_sort, "combine": _plain_combine, "grad": _plain_grad, "product": _plain_product}[op](state)


def _run_sort(s):
    import quantized_routed_expert_noaux_b200 as q
    c = s["case"]
    act = q.COLI_ACT_F32 if c["dtype"] == "f32" else q.COLI_ACT_BF16
    q.coli_moe_sort_rows(c["experts"], c["top_k"], act, s["x"], c["tokens"], c["hidden"], c["hidden"], s["ids"], s["offsets"],
                         s["perm"], s["place"], s["rows"], c["hidden"], s["ws"])
    return {"offsets": s["offsets"], "perm": s["perm"], "place": s["place"], "rows": s["rows"]}


def _run_combine(s):
    import quantized_routed_expert_noaux_b200 as q
    c = s["case"]
    act, out = (q.COLI_ACT_F32 if c[v] == "f32" else q.COLI_ACT_BF16 for v in ("dtype", "out"))
    q.coli_moe_combine(act, s["y"], s["y"].shape[0], c["hidden"], s["place"], s["w"], c["tokens"], c["top_k"], c["hidden"], out,
                       s["add"], c["hidden"], s["out"], c["hidden"], s["ws"])
    return s["out"]


def _run_grad(s):
    import quantized_routed_expert_noaux_b200 as q
    c = s["case"]
    act, out = (q.COLI_ACT_F32 if c[v] == "f32" else q.COLI_ACT_BF16 for v in ("dtype", "out"))
    q.coli_moe_combine_grad(act, s["y"], s["y"].shape[0], c["hidden"], s["place"], s["w"], c["tokens"], c["top_k"], c["hidden"], out,
                            s["dout"], c["hidden"], s["dy"], c["hidden"], s["dw"], s["ws"])
    return {"dy": s["dy"], "dw": s["dw"]}


def _run_product(s):
    import quantized_routed_expert_noaux_b200 as q
    c = s["case"]
    x, codes = s["x"], s["codes"]
    q.coli_moe_i8_quantize(q.COLI_ACT_F32 if c["dtype"] == "f32" else q.COLI_ACT_BF16, int(c["glu"]), x, x.shape[0], x.shape[1], c["k"],
                           s["place"], c["top_k"] if s["place"] is not None else 1, codes.shape[0], codes, codes.shape[1], s["scale"], s["ws"])
    q.coli_moe_i8_product(q.i8_rows_for(codes, s["scale"]), q.i8_mats_for(s["wc"], s["wscale"]), c["k"], s["offsets"],
                          q.COLI_ACT_F32 if c["out"] == "f32" else q.COLI_ACT_BF16, s["out"], c["n"], s["ws"])
    return s["out"]


def _plain_sort(s):
    c = s["case"]
    ids = s["ids"].reshape(-1).long()
    key = torch.where(ids < 0, c["experts"], ids)
    order, perm = torch.sort(key, stable=True)
    place = torch.empty_like(perm)
    place[perm] = torch.arange(perm.numel(), device=perm.device)
    offsets = torch.searchsorted(order, torch.arange(c["experts"] + 1, device=perm.device))
    live = order < c["experts"]
    rows = torch.where(live[:, None], s["x"][torch.div(perm, c["top_k"], rounding_mode="floor")], 0.0)
    return {"offsets": offsets.to(torch.int32), "perm": torch.where(live, perm, -1).to(torch.int32),
            "place": torch.where(ids < 0, -1, place).to(torch.int32), "rows": rows.to(s["x"].dtype)}


def _plain_combine(s):
    place = s["place"].long()
    live = place >= 0
    v = s["y"][place.clamp(min=0)].to(torch.float32)
    f = live.to(torch.float32) if s["w"] is None else torch.where(live, s["w"], 0.0)
    total = (v * f[:, :, None]).sum(1)
    if s["add"] is not None:
        total = total + s["add"].to(torch.float32)
    return total.to(s["out"].dtype)


def _plain_grad(s):
    place = s["place"].long()
    live = place >= 0
    d = s["dout"].to(torch.float32)[:, None, :]
    dw = torch.where(live, (s["y"][place.clamp(min=0)].to(torch.float32) * d).sum(2), 0.0)
    # one row more, for the slots that have none
    rows = s["dy"].shape[0]
    dy = torch.zeros(rows + 1, s["dy"].shape[1], device=d.device)
    dy[torch.where(live, place, rows)] = d * s["w"][:, :, None]
    return {"dy": dy[:rows].to(s["dy"].dtype), "dw": dw}


def _plain_product(s):
    c = s["case"]
    k, rows = c["k"], s["codes"].shape[0]
    # in 64 bits: which code is the nearest is decided by the last bits
    x = s["x"].double()
    if c["glu"]:
        x = x[:, :k] / (1 + torch.exp(-x[:, :k])) * x[:, k:]
    top = x.abs().amax(1, keepdim=True)
    codes = torch.round(x * 127 / top).to(torch.float32)
    scale = (top / 127).to(torch.float32)
    if s["place"] is not None:
        slot = torch.empty(rows, dtype=torch.long, device=x.device)
        slot[s["place"].long()] = torch.arange(rows, device=x.device)
        source = torch.div(slot, c["top_k"], rounding_mode="floor")
        codes, scale = codes[source], scale[source]
    w = s["wc"][:, :, :k].to(torch.float32)
    if s["offsets"] is None:
        return (torch.matmul(codes, w[0].t()) * scale * s["wscale"][0]).to(s["out"].dtype)
    # every expert's rows side by side in one batch, as many as the fullest one has
    off = s["offsets"].long()
    at = torch.arange(rows, device=x.device)
    expert = torch.searchsorted(off[1:], at, right=True)
    nth = at - off[expert]
    batch = torch.zeros(c["experts"], s["fullest"], k, device=x.device)
    batch[expert, nth] = codes
    sums = torch.bmm(batch, w.transpose(1, 2))[expert, nth]
    return (sums * scale * s["wscale"][expert]).to(s["out"].dtype)


# ------------------------------------------------------------------ 64-bit results


def _exact_sort(s):
    c = s["case"]
    flat = s["ids"].reshape(-1)
    rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=flat.device)
    slots = torch.cat([torch.nonzero(flat == e)[:, 0] for e in range(c["experts"])])
    rows[:slots.numel()] = s["x"].double().index_select(0, slots // c["top_k"])
    return {"offsets": None, "perm": None, "place": None, "rows": rows}


def _exact_combine(s):
    c = s["case"]
    total = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device="cuda")
    if s["add"] is not None:
        total += s["add"]
    for j in range(c["top_k"]):
        at = s["place"][:, j]
        have = (at >= 0).nonzero()[:, 0]
        term = s["y"].index_select(0, at[have].long()).double()
        if s["w"] is not None:
            term = term * s["w"][have, j].double()[:, None]
        total.index_add_(0, have, term)
    return total


def _exact_grad(s):
    c = s["case"]
    d = s["dout"].double()
    dy = torch.zeros(s["dy"].shape, dtype=torch.float64, device=d.device)
    dw = torch.zeros(c["tokens"], c["top_k"], dtype=torch.float64, device=d.device)
    for j in range(c["top_k"]):
        have = (s["place"][:, j] >= 0).nonzero()[:, 0]
        at = s["place"][have, j].long()
        dw[have, j] = torch.einsum("th,th->t", d[have], s["y"][at].double())
        dy[at] = d[have] * s["w"][have, j].double()[:, None]
    return {"dy": dy, "dw": dw}


def _exact_product(s):
    c = s["case"]
    k = c["k"]
    v = s["x"].to(torch.float64)
    if c["glu"]:
        gate, up = v.split(k, 1)
        v = gate * torch.sigmoid(gate) * up
    top = v.abs().max(1, keepdim=True).values
    v = torch.round(v * 127 / top) * (top / 127)
    if s["place"] is not None:
        slots = torch.empty_like(s["place"], dtype=torch.long)
        slots.scatter_(0, s["place"].long(), torch.arange(slots.numel(), device=slots.device) // c["top_k"])
        v = v.index_select(0, slots)
    ends = [0, v.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    parts = []
    for i, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if hi > lo:
            m = s["wc"][i].narrow(1, 0, k).double() * s["wscale"][i].double()[:, None]
            parts.append(v[lo:hi] @ m.t())
    return torch.cat(parts)


def exact(case, seed):
    s = prepare(case, seed)
    return {"sort": _exact_sort, "combine": _exact_combine, "grad": _exact_grad, "product": _exact_product}[case["op"]](s)
