"""The layer over records in microscaled 4-bit containers: packing, the expert half against plain 64-bit
arithmetic, and the whole layer with its routing."""
import numpy as np
import pytest
import torch

import _fp4 as ref
import synth

q = pytest.importorskip("quantized_routed_expert_noaux_b200")

FMT = {20: 1, 36: 0}


def config(wfmt, H=256, I=128, E=8, K=3, shared=1, act=1):
    return q.MoEConfig(H, I, E, K, 1, 1, shared, I, 2.5, wfmt, act, 0)


def bf16(v):
    return torch.from_numpy(np.asarray(v, np.float64)).to(torch.bfloat16).double().numpy()


class Experts:
    """E records and a shared one from random matrices, on the device, with the values they stand for."""

    def __init__(self, cfg, seed=0):
        g = torch.Generator().manual_seed(seed)
        H, I, E = cfg.hidden, cfg.inter, cfg.n_experts
        self.cfg, self.fmt = cfg, FMT[cfg.wfmt]
        n = q.coli_moe_record_bytes(H, I, cfg.wfmt)
        stride = (n + 255) // 256 * 256
        self.recs = torch.zeros(E + 1, stride, dtype=torch.uint8, device="cuda")
        self.ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
        self.mats = []
        for e in range(E + 1):
            wg, wu, wd = (torch.randn(r, c, generator=g) * 0.1 for r, c in ((I, H), (I, H), (H, I)))
            q.coli_moe_fp4_pack_record(cfg, 0, wg.cuda(), wu.cuda(), wd.cuda(), self.recs[e], self.ws)
            self.mats.append((wg, wu, wd))
        self.values = [tuple(ref.values(*ref.quantize(m.numpy(), self.fmt), self.fmt) for m in ms) for ms in self.mats]
        self.Wr = (torch.randn(E, H, generator=g) / H ** 0.5).cuda()
        self.bias = (torch.randn(E, generator=g) * 0.1).cuda()
        self.weights = q.weights_for(self.Wr, self.bias, self.recs[:E], self.recs[E] if cfg.n_shared else None)

    def expert(self, x64, e):
        """(y, tolerance of y) [T, H] of expert e for rows x64 (float64, before quantisation)."""
        H, I = self.cfg.hidden, self.cfg.inter
        wg, wu, wd = self.values[e]
        xq = ref.values(*ref.quantize(x64, self.fmt), self.fmt)
        g, u = xq @ wg.T, xq @ wu.T
        # float32 sums of H terms: a unit of 2^-23 of the largest partial sum for each term at most
        dg = H * 2.0 ** -23 * (np.abs(xq) @ np.abs(wg).T)
        du = H * 2.0 ** -23 * (np.abs(xq) @ np.abs(wu).T)
        h = g / (1 + np.exp(-g)) * u
        # |d silu/dg| <= 1.1; expf and three more roundings
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(g) * du + 8 * 2.0 ** -24 * np.abs(h)
        h0, hi, lo = (ref.values(*ref.quantize(bf16(v), self.fmt), self.fmt) for v in (h, h + dh, h - dh))
        # what a sum off by dh can make of the 4-bit value (twice: scale and code may move apart)
        dq = 2 * np.maximum(np.abs(hi - h0), np.abs(lo - h0))
        y = h0 @ wd.T
        tol = dq @ np.abs(wd).T + I * 2.0 ** -23 * (np.abs(h0) @ np.abs(wd).T)
        return y, tol + 2.0 ** -8 * 1.01 * (np.abs(y) + tol)   # rounded to bf16

    def ffn(self, x64, ids, w):
        """Result and tolerance of the expert half for a routing."""
        T, K = ids.shape
        out, tol = np.zeros((T, self.cfg.hidden)), np.zeros((T, self.cfg.hidden))
        for e in range(self.cfg.n_experts):
            t, k = np.nonzero(ids == e)
            if len(t):
                y, d = self.expert(x64[t], e)
                np.add.at(out, t, w[t, k][:, None] * y)
                np.add.at(tol, t, w[t, k][:, None] * (d + (K + 1) * 2.0 ** -24 * np.abs(y)))
        if self.cfg.n_shared:
            y, d = self.expert(x64, self.cfg.n_experts)
            out, tol = out + y, tol + d + (K + 1) * 2.0 ** -24 * np.abs(y)
        return out, tol + (K + 2) * 2.0 ** -24 * np.abs(out)


@pytest.mark.gpu
@pytest.mark.parametrize("wfmt", [20, 36])
@pytest.mark.parametrize("act", [0, 1])
def test_pack_record(wfmt, act):
    """A record is the two quantised matrices, gate and up rows in runs of 16."""
    H, I = 192, 64
    cfg, fmt = config(wfmt, H, I), FMT[wfmt]
    g = torch.Generator().manual_seed(4)
    ms = [(torch.randn(r, c, generator=g)).to(torch.float32 if act == 0 else torch.bfloat16) for r, c in ((I, H), (I, H), (H, I))]
    n = q.coli_moe_record_bytes(H, I, wfmt)
    rec = torch.full(((n + 255) // 256 * 256,), 0xA5, dtype=torch.uint8, device="cuda")
    q.coli_moe_fp4_pack_record(cfg, act, *[m.cuda() for m in ms], rec, torch.zeros(512, dtype=torch.uint8, device="cuda"))
    wg, wu, wd = (m.double().numpy() for m in ms)
    w1 = np.stack([wg.reshape(-1, 16, H), wu.reshape(-1, 16, H)], 1).reshape(2 * I, H)
    c1, b1, r1 = ref.quantize(w1, fmt)
    cd, bd, rd = ref.quantize(wd, fmt)
    parts = [ref.pack(c1), ref.pack(cd), ref.tiles_layout(b1, fmt, H), ref.tiles_layout(bd, fmt, I)]
    if fmt == 1:
        parts += [r1.view(np.uint8), rd.view(np.uint8)]
    want = np.concatenate([p.reshape(-1) for p in parts])
    assert len(want) == n
    got = rec.cpu().numpy()
    assert np.array_equal(got[:n], want) and (got[n:] == 0xA5).all()


def group(cfg, ids, T, ws):
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    E, K = cfg.n_experts, cfg.top_k
    arrays = i32(E), i32(E + 1), i32(T * K), i32(E), i32(1)
    q.coli_moe_group(cfg, ids, T, *arrays, ws)
    return arrays


@pytest.mark.gpu
@pytest.mark.parametrize("wfmt", [20, 36])
@pytest.mark.parametrize("T,H,I,E,K,shared,act", [(1, 256, 128, 8, 3, 1, 1), (3, 192, 320, 5, 2, 0, 0), (17, 256, 64, 16, 4, 1, 0),
                                                  (90, 320, 192, 4, 2, 1, 1), (300, 256, 192, 2, 2, 1, 1), (5, 256, 128, 64, 8, 1, 1), (3, 64, 64, 1024, 8, 1, 1)])
def test_expert_half(wfmt, T, H, I, E, K, shared, act):
    cfg = config(wfmt, H, I, E, K, shared, act)
    ex = Experts(cfg)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).to(torch.float32 if act == 0 else torch.bfloat16)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(torch.int32)
    w = torch.rand(T, K, generator=g)
    ws = torch.full((q.coli_moe_workspace_size(cfg, T),), 0xFF, dtype=torch.uint8, device="cuda")  # nothing may rely on its contents
    q.coli_moe_clear_error(ws)
    counts, offsets, perm, uniq, nu = group(cfg, ids.cuda(), T, ws)
    out = torch.full((T, H), -7.0, device="cuda")
    q.coli_moe_ffn(cfg, ex.weights, x.cuda(), T, w.cuda(), offsets, perm, uniq, nu, out, ws)
    assert q.coli_moe_error_word(ws) == 0
    want, tol = ex.ffn(x.double().numpy(), ids.numpy(), w.double().numpy())
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
    # the tolerance can tell a wrong row, scale or expert from a right one: those are off by the result's own
    # size, and the tolerance is a small part of it.  Its parts: 2^-8 of the sum of the terms' sizes, about
    # twice the result's (1%); 4-bit steps that may flip: dh is about 4e-4 of h at H = 256, so 4e-4 / 2^-7 of
    # the bf16 roundings (5%) and 2^-7 / (1/4) of those (3%), 0.2% of the elements, by up to a third, twice,
    # their sizes added up over I terms against a sum that grows with sqrt(I): 0.13% * sqrt(320) (2%)
    assert np.linalg.norm(tol) < 0.25 * np.linalg.norm(want)
    again = torch.empty_like(out)
    q.coli_moe_ffn(cfg, ex.weights, x.cuda(), T, w.cuda(), offsets, perm, uniq, nu, again, ws)
    assert torch.equal(out, again)


@pytest.mark.gpu
@pytest.mark.parametrize("wfmt", [20, 36])
@pytest.mark.parametrize("T,act", [(1, 1), (6, 0), (64, 1), (65, 0), (130, 1)])
def test_whole_layer(wfmt, T, act):
    """The layer is its parts: routing as coli_moe_route_scores gives it (and coli_moe_route, but for the last
    bits of its weights), the expert half on that routing, bit for bit; replayed from a graph with new
    activations too; and without allocation."""
    cfg = config(wfmt, act=act)
    assert q.coli_moe_layer_kernels(cfg, T) == 8
    ex = Experts(cfg)
    H, K = cfg.hidden, cfg.top_k
    g = torch.Generator().manual_seed(T)
    xs = [torch.randn(T, H, generator=g).to(torch.bfloat16 if act else torch.float32).cuda() for _ in range(2)]
    ws = torch.zeros(q.coli_moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    ids, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")

    def parts(x):
        logits = torch.empty(T, cfg.n_experts, device="cuda")
        i, v, out = torch.empty_like(ids), torch.empty_like(w), torch.empty(T, H, device="cuda")
        q.coli_moe_gate(cfg, ex.Wr, x, T, logits)
        q.coli_moe_route(cfg, logits, ex.bias, T, i, v)
        i0, v0 = i.clone(), v.clone()
        q.coli_moe_route_scores(q.MoERouter(cfg.n_experts, K, cfg.n_group, cfg.topk_group, q.COLI_SCORE_SIGMOID, q.COLI_GROUP_TOP2, 1, 0,
                                            cfg.routed_scaling), logits, 0, ex.bias, T, i, v)
        assert torch.equal(i, i0) and torch.allclose(v, v0, rtol=(cfg.n_experts + 8) * 2.0 ** -24, atol=0)
        # the gate's sums are double: its float32 logits are the exact dot products' roundings, or a neighbour's
        exact = x.double() @ ex.Wr.double().T
        assert (torch.abs(logits.double() - exact) <= 2.0 ** -24 * 1.001 * exact.abs() + 1e-12).all()
        _, offsets, perm, uniq, nu = group(cfg, i, T, ws)
        q.coli_moe_ffn(cfg, ex.weights, x, T, v, offsets, perm, uniq, nu, out, ws)
        return i, v, out

    x, out = xs[0].clone(), torch.empty(T, H, device="cuda")
    q.coli_moe_layer(cfg, ex.weights, x, T, out, ids, w, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.coli_moe_layer(cfg, ex.weights, x, T, out, ids, w, ws)
    for new in xs:
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert q.coli_moe_error_word(ws) == 0
        i, v, o = parts(new)
        assert torch.equal(ids, i) and torch.equal(w, v) and torch.equal(out, o)
    if q.coli_moe_workspace_size(cfg, T) <= q.STATIC_SCRATCH_BYTES:
        o2 = torch.empty_like(out)
        q.coli_moe_layer_noalloc(cfg, ex.weights, x, T, o2)
        assert torch.equal(out, o2) and q.coli_moe_noalloc_error_word() == 0


@pytest.mark.gpu
def test_softmax_router_in_front_of_the_experts():
    """gate -> softmax routing -> group -> expert half: a layer of another routing family, with a padded
    token whose logits are masked."""
    cfg = config(20, E=16, K=4)
    ex = Experts(cfg, 2)
    T, H, E, K = 9, cfg.hidden, 16, 4
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    xd = x.cuda()
    ws = torch.zeros(q.coli_moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    logits = torch.empty(T, E, device="cuda")
    q.coli_moe_gate(cfg, ex.Wr, xd, T, logits)
    logits[8] = float("-inf")
    ids, w = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    q.coli_moe_route_scores(q.MoERouter(E, K, 1, 1, q.COLI_SCORE_SOFTMAX, q.COLI_GROUP_MAX, 1, 0, 1.0), logits, 0, None, T, ids, w)
    _, offsets, perm, uniq, nu = group(cfg, ids, T, ws)
    out = torch.empty(T, H, device="cuda")
    q.coli_moe_ffn(cfg, ex.weights, xd, T, w, offsets, perm, uniq, nu, out, ws)
    assert q.coli_moe_error_word(ws) == 0
    assert torch.allclose(w[:8].sum(1), torch.ones(8, device="cuda"), rtol=1e-6) and (w[8] == 0).all()
    want, tol = ex.ffn(x.double().numpy(), ids.cpu().numpy(), w.double().cpu().numpy())
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.gpu
def test_bad_ids_are_left_out():
    """Slots with an id outside [0, E) add nothing and set the error word; the others stand."""
    cfg = config(36, E=4, K=2)
    ex = Experts(cfg)
    T, H = 5, cfg.hidden
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    ids = torch.tensor([[0, 1], [3, -1], [7, 2], [1, 0], [2, 3]], dtype=torch.int32)
    w = torch.ones(T, 2)
    ws = torch.zeros(q.coli_moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    _, offsets, perm, uniq, nu = group(cfg, ids.cuda(), T, ws)
    out = torch.empty(T, H, device="cuda")
    q.coli_moe_ffn(cfg, ex.weights, x.cuda(), T, w.cuda(), offsets, perm, uniq, nu, out, ws)
    assert q.coli_moe_error_word(ws) & q.DEVERR_EXPERT_ID
    want, tol = ex.ffn(x.double().numpy(), ids.numpy(), w.double().numpy())
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_configs_on_the_host():
    for wfmt in (20, 36):
        cfg = config(wfmt, 6144, 2048, 256, 8)
        q.coli_moe_check_config(cfg)
        assert q.coli_moe_layer_kernels(cfg, 1) == q.coli_moe_layer_kernels(cfg, 4096) == 8
        assert q.coli_moe_layer_kernels(cfg, 0) == 0
        # codes, scales, row scales of 3 x 2048 x 6144 values
        per = 16 if wfmt == 20 else 32
        rows = (2 * 2048 + 6144) * 4 if wfmt == 20 else 0
        assert q.coli_moe_record_bytes(6144, 2048, wfmt) == 3 * 2048 * 6144 // 2 + 3 * 2048 * 6144 // per + rows
        for field, value, status in (("group_size", 64, 4), ("hidden", 100, 2), ("inter", 96, 2)):
            bad = config(wfmt, 6144, 2048, 256, 8, shared=0)
            setattr(bad, field, value)
            with pytest.raises(q.ColiError) as ei:
                q.coli_moe_check_config(bad)
            assert ei.value.status == status
        with pytest.raises(q.ColiError) as ei:
            q.coli_moe_record_bytes(6144, 96, wfmt)
        assert ei.value.status == 2


def test_pack_record_refusals():
    def refused(status, cfg, *args):
        with pytest.raises(q.ColiError) as ei:
            q.coli_moe_fp4_pack_record(cfg, *args, stream=0)
        assert ei.value.status == status
    cfg = config(20)
    refused(4, q.config_for(synth.WORKLOADS["tiny"]), 0, 256, 512, 1024, 2048, 4096)
    refused(1, cfg, 2, 256, 512, 1024, 2048, 4096)
    refused(1, cfg, 0, 256, None, 1024, 2048, 4096)
    refused(3, cfg, 0, 264, 512, 1024, 2048, 4096)
    refused(3, cfg, 0, 256, 512, 1024, 2064, 4096)
    refused(7, cfg, 0, 256, 512, 1024, 2048, None)
