"""Routing from scores (coli_moe_route_scores) against a plain 64-bit implementation, one token at a time."""
import math

import numpy as np
import pytest
import torch

q = pytest.importorskip("quantized_routed_expert_noaux_b200")

SIG, SOFT, TOP2, MAXG = 0, 1, 0, 1
INF = float("inf")


def router(E, K, G=1, TG=1, score=SOFT, group=MAXG, renorm=1, act=0, scaling=1.0):
    return q.MoERouter(E, K, G, TG, score, group, renorm, act, scaling)


def one_token(l, bias, r):
    """ids and float64 weights of one row of float64 logits."""
    E, K, G = r.n_experts, r.top_k, r.n_group
    live = [e for e in range(E) if l[e] > -INF]
    if r.score == SOFT:
        top = max((l[e] for e in live), default=0.0)
        ex = [0.0] * E
        for e in live:
            ex[e] = 1.0 if l[e] == top else math.exp(l[e] - top)
        total = math.fsum(ex)
        s = [v / total if total else 0.0 for v in ex]
    else:
        s = [0.0 if not l[e] > -INF else (1.0 / (1.0 + math.exp(-l[e])) if l[e] > -700 else 0.0) for e in range(E)]
    rank = [l[e] if bias is None else s[e] + bias[e] for e in range(E)]
    by = s if bias is None else rank
    ok = [e for e in live if rank[e] > -INF]
    if r.topk_group < G:
        gs = E // G
        best = []
        for g in range(G):
            mem = [e for e in ok if e // gs == g]
            if not mem:
                best.append(-INF)
            elif r.group_score == MAXG:
                best.append(max(rank[e] for e in mem))
            else:
                best.append(sum(sorted((by[e] for e in mem), reverse=True)[:2]))
        has = [any(e // gs == g for e in ok) for g in range(G)]
        kept = sorted(range(G), key=lambda g: (not has[g], -best[g], g))[:r.topk_group]
        ok = [e for e in ok if e // gs in kept]
    ids = sorted(ok, key=lambda e: (-rank[e], e))[:K]
    if r.score == SOFT and r.renorm and ids:
        ref = max(l[e] for e in ids)
        w = [1.0 if l[e] == ref else math.exp(l[e] - ref) for e in ids]
    else:
        w = [s[e] for e in ids]
    if r.renorm:
        d = sum(w)
        w = [v / d if d else 0.0 for v in w]
    w = [v * r.scaling for v in w] + [0.0] * (K - len(ids))
    ids += [e for e in range(E) if e not in ids][:K - len(ids)]
    return ids, w


def check(logits, bias, r, ld=0, T=None):
    """logits: 2-d host tensor [T, E]; ld > E spreads the rows."""
    T = logits.shape[0]
    E, K = r.n_experts, r.top_k
    dev = logits
    if ld:
        dev = torch.full((T, ld), float("nan"), dtype=logits.dtype)
        dev[:, :E] = logits
    dev = dev.cuda()
    ids = torch.full((T, K), -5, dtype=torch.int32, device="cuda")
    w = torch.full((T, K), -7.0, device="cuda")
    q.coli_moe_route_scores(r, dev, ld, None if bias is None else bias.cuda(), T, ids, w)
    ids, w = ids.cpu().numpy(), w.cpu().double().numpy()
    l64 = logits.double().numpy()
    b64 = None if bias is None else bias.double().numpy()
    for t in range(T):
        want_ids, want_w = one_token(l64[t].tolist(), None if b64 is None else b64.tolist(), r)
        assert ids[t].tolist() == want_ids, t
        # float32 exp (2 ulp) and sums of E terms, a quotient and two products: (E + 8) half units in the last
        # place; a softmax weight of a logit far below the row's largest may leave float32's range
        tol = (r.n_experts + 8) * 2.0 ** -24 * np.abs(want_w) + 2.0 ** -126
        assert (np.abs(w[t] - want_w) <= tol).all(), (t, w[t], want_w)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("T,E,K,G,TG,group,renorm", [
    (1, 256, 8, 8, 4, TOP2, 1), (5, 64, 8, 1, 1, MAXG, 1), (33, 256, 8, 8, 3, MAXG, 0), (7, 1024, 32, 32, 5, TOP2, 1),
    (9, 40, 6, 5, 2, TOP2, 0), (6, 96, 16, 3, 2, MAXG, 1), (4, 1, 1, 1, 1, MAXG, 1), (4, 33, 32, 1, 1, TOP2, 0),
    (3, 1000, 10, 4, 1, TOP2, 1), (3, 8, 2, 8, 3, TOP2, 1), (3, 130, 5, 26, 7, MAXG, 0), (130, 17, 3, 1, 1, MAXG, 0),
])
def test_route_scores(score, biased, act, T, E, K, G, TG, group, renorm):
    g = torch.Generator().manual_seed(E * 3 + T)
    logits = (torch.randn(T, E, generator=g) * 2).to(torch.float32 if act == 0 else torch.bfloat16)
    bias = torch.randn(E, generator=g) * 0.1 if biased else None
    r = router(E, K, G, TG, score, group, renorm, act, 2.5)
    check(logits, bias, r)
    check(logits[:3], bias, r, ld=E + 5)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group", [TOP2, MAXG])
def test_ties_and_masks(score, biased, group):
    """Equal logits, experts masked by -inf and NaN, rows without any expert, infinite logits, biases of
    -inf, signed zeros, saturated scores."""
    E = 32
    g = torch.Generator().manual_seed(5)
    l = torch.randint(-2, 3, (16, E), generator=g).float()      # many ties
    l[1] = 0.0
    l[1, ::2] = -0.0
    l[2] = -INF
    l[3] = float("nan")
    l[4] = -INF
    l[4, 30] = 0.5                                               # fewer than K
    l[5, :24] = -INF                                             # whole groups masked
    l[6, 7] = INF
    l[7, [3, 9, 21]] = INF
    l[8] = torch.where(torch.rand(E, generator=g) < 0.7, torch.tensor(float("nan")), l[8])
    l[9] = 100.0 + torch.arange(E)                               # sigmoid saturates, softmax does not
    l[10] = -100.0 - torch.arange(E)
    l[11] = -3.0e38
    l[12] = 3.0e38
    bias = torch.randint(-1, 2, (E,), generator=g).float() * 0.25 if biased else None
    for renorm in (0, 1):
        for G, TG, K in ((1, 1, 6), (4, 2, 6), (8, 1, 4), (4, 4, 32)):
            check(l, bias, router(E, K, G, TG, score, group, renorm))
            if biased:
                b2 = bias.clone()
                b2[[0, 5, 6, 31]] = -INF
                b2[7] = float("nan")
                check(l, b2, router(E, K, G, TG, score, group, renorm))


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("E,G,TG,K", [(256, 8, 4, 8), (64, 1, 1, 6), (1024, 16, 2, 32), (40, 5, 2, 3)])
@pytest.mark.parametrize("group", [TOP2, MAXG])
def test_scores_closer_than_float32(score, E, G, TG, K, group):
    """Biases that bring every s + b to within float32's last bits of one value: the choice between
    experts and between groups is double's; some tokens have clear experts beside them."""
    g = torch.Generator().manual_seed(E)
    l = torch.randn(1, E, generator=g)
    l64 = l.double()
    s = torch.softmax(l64, 1)[0] if score == SOFT else torch.sigmoid(l64)[0]
    bias = (0.75 - s).float()
    rows = l.repeat(6, 1)
    rows[1, ::7] += 1e-6
    rows[2] = l[0].flip(0)
    rows[4, :: E // G] += 3.0
    check(rows, bias, router(E, K, G, TG, score, group, 1))
    check(rows, torch.zeros(E), router(E, K, G, TG, score, group, 0))


@pytest.mark.gpu
def test_every_row_can_be_grouped():
    """Masked rows still hold K different ids, so the batch goes on through coli_moe_group."""
    import synth
    cfg = q.config_for(synth.WORKLOADS["tiny"])
    E, K, T = cfg.n_experts, cfg.top_k, 9
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(1))
    l[3], l[5] = float("nan"), -INF
    l[6, 2:] = -INF
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    w = torch.empty(T, K, device="cuda")
    q.coli_moe_route_scores(router(E, K), l.cuda(), 0, None, T, ids, w)
    ws = torch.zeros(q.coli_moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, perm, uniq, nu = i32(E), i32(E + 1), i32(T * K), i32(E), i32(1)
    q.coli_moe_group(cfg, ids, T, counts, offsets, perm, uniq, nu, ws)
    assert q.coli_moe_error_word(ws) == 0
    assert int(offsets[-1]) == T * K
    assert (w[[3, 5]] == 0).all() and torch.equal(ids[3].cpu(), torch.arange(K, dtype=torch.int32))
    assert ids[6, :2].sort().values.tolist() == [0, 1] and (w[6, 2:] == 0).all()


@pytest.mark.gpu
def test_replayed_from_a_graph():
    T, E = 24, 64
    r = router(E, 8, score=SIG)
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(2))
    dev = l.cuda()
    ids, w = torch.empty(T, 8, dtype=torch.int32, device="cuda"), torch.empty(T, 8, device="cuda")
    q.coli_moe_route_scores(r, dev, 0, None, T, ids, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.coli_moe_route_scores(r, dev, 0, None, T, ids, w)
    dev.copy_(l.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    for t in range(T):
        assert ids[t].tolist() == one_token(l.flip(0)[t].double().tolist(), None, r)[0]


@pytest.mark.parametrize("field,value,status", [
    ("score", 2, 1), ("group_score", -1, 1), ("renorm", 2, 1), ("logits", 2, 1), ("scaling", 0.0, 1), ("scaling", float("nan"), 1),
    ("n_experts", 0, 2), ("n_experts", 2048, 4), ("top_k", 0, 2), ("top_k", 33, 4), ("top_k", 129, 2), ("n_group", 7, 2),
    ("topk_group", 9, 2), ("n_group", 64, 4),
])
def test_bad_routers_are_refused(field, value, status):
    r = router(256, 8, 8, 4)
    q.coli_moe_check_router(r)
    setattr(r, field, value)
    if field == "n_group" and value == 64:
        r.topk_group, r.top_k = 64, 8
    with pytest.raises(q.ColiError) as ei:
        q.coli_moe_check_router(r)
    assert ei.value.status == status


def test_bad_calls_are_refused():
    r = router(64, 8)

    def refused(status, *args):
        with pytest.raises(q.ColiError) as ei:
            q.coli_moe_route_scores(r, *args, stream=0)
        assert ei.value.status == status
    refused(2, 256, 0, None, -1, 512, 1024)
    refused(2, 256, 63, None, 4, 512, 1024)
    refused(4, 256, 0, None, (1 << 30) + 1, 512, 1024)
    refused(1, None, 0, None, 4, 512, 1024)
    refused(1, 256, 0, None, 4, None, 1024)
    refused(1, 256, 0, None, 4, 512, None)
    refused(3, 258, 0, None, 4, 512, 1024)
    refused(3, 256, 0, 513, 4, 512, 1024)
    q.coli_moe_route_scores(r, None, 0, None, 0, None, None, stream=0)  # no tokens: a no-op
