"""Slots sorted by expert with their rows, the weighted sum back and its gradient, against plain 64-bit arithmetic.

Sorting and copying are exact.  A sum of n float32 terms, added one by one with one rounding each, is within n * 2^-24 of
the sum of their magnitudes; a result in bf16 is rounded once more, by at most 2^-8 of itself."""
import numpy as np
import pytest
import torch

q = pytest.importorskip("quantized_routed_expert_noaux_b200")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACT = {"f32": 0, "bf16": 1}


def ws():
    return torch.zeros(512, dtype=torch.uint8, device="cuda")


def refused(status, fn, *args, **kw):
    with pytest.raises(q.ColiError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status


def rows_at(values, ld, off, dtype):
    """`values` [n, h] as a device view whose rows lie ld elements apart, `off` elements into its storage, NaN around."""
    n, h = values.shape
    flat = torch.full((off + max(n, 1) * ld + 16,), float("nan"), dtype=DT[dtype], device="cuda")
    view = flat[off:off + max(n, 1) * ld].view(max(n, 1), ld)[:n, :h]
    view.copy_(values)
    return flat, view


# ------------------------------------------------------------------ refusals (host)


def test_refusals():
    """Pointers stand for device memory that no call reaches: every one of these ends before a launch."""
    S = [8, 2, 0, 256, 3, 16, 16, 256, 256, 256, 256, 256, 16, 256]

    def sort(status, **kw):
        names = ["n_experts", "top_k", "act", "x", "T", "hidden", "ldx", "topk_ids", "offsets", "perm", "place", "rows", "ldr", "ws"]
        refused(status, q.coli_moe_sort_rows, *[kw.get(n, v) for n, v in zip(names, S)], stream=0)
    sort(1, act=2)
    sort(1, x=None)
    sort(1, rows=None)
    sort(1, topk_ids=None)
    sort(1, offsets=None)
    sort(1, perm=None)
    sort(1, place=None)
    sort(2, T=-1)
    sort(2, top_k=0)
    sort(2, hidden=0)
    sort(2, n_experts=0)
    sort(2, ldx=15)
    sort(2, ldr=15)
    sort(4, n_experts=1025)
    sort(4, top_k=33)
    sort(4, hidden=(1 << 20) + 1, ldx=1 << 21, ldr=1 << 21)
    sort(4, T=(1 << 29) + 1)
    sort(3, x=258)
    sort(3, act=1, rows=257)
    sort(3, place=258)
    sort(7, ws=None)
    sort(7, ws=128)
    C = [0, 256, 4, 16, 256, 256, 3, 2, 16, 0, 256, 16, 256, 16, 256]

    def combine(status, **kw):
        names = ["act", "y", "rows", "ldy", "place", "topk_w", "T", "top_k", "hidden", "out_type", "add", "ld_add", "out", "ldo", "ws"]
        refused(status, q.coli_moe_combine, *[kw.get(n, v) for n, v in zip(names, C)], stream=0)
    combine(1, act=-1)
    combine(1, out_type=2)
    combine(1, y=None)
    combine(1, place=None)
    combine(1, out=None)
    combine(2, rows=-1)
    combine(2, ldy=15)
    combine(2, ldo=15)
    combine(2, ld_add=15)
    combine(2, hidden=0)
    combine(4, top_k=33)
    combine(3, y=258)
    combine(3, out_type=1, add=257)
    combine(3, topk_w=258)
    combine(7, ws=None)
    G = [0, 256, 4, 16, 256, 256, 3, 2, 16, 0, 256, 16, 256, 16, 256, 256]

    def grad(status, **kw):
        names = ["act", "y", "rows", "ldy", "place", "topk_w", "T", "top_k", "hidden", "out_type", "dout", "ld_dout", "dy", "ld_dy", "dw", "ws"]
        refused(status, q.coli_moe_combine_grad, *[kw.get(n, v) for n, v in zip(names, G)], stream=0)
    grad(1, act=3)
    grad(1, dout=None)
    grad(1, place=None)
    grad(1, y=None)
    grad(1, dy=None, dw=None)
    grad(2, ldy=15)
    grad(2, ld_dout=15)
    grad(2, ld_dy=15)
    grad(4, T=1 << 30)
    grad(3, dw=257)
    grad(3, dy=258)
    grad(7, ws=64)


@pytest.mark.parametrize("explicit", [False, True])
def test_any_tensor_off_the_gpu_is_refused(explicit):
    if torch.cuda.is_available():
        pytest.skip("host check: where it runs nothing could be launched on such a pointer")
    kw = {"stream": 0} if explicit else {}
    t = torch.zeros(64)
    for fn, args, places in ((q.coli_moe_sort_rows, [8, 2, 0, 256, 3, 16, 16, 256, 256, 256, 256, 256, 16, 256], (3, 7, 8, 9, 10, 11, 13)),
                             (q.coli_moe_combine, [0, 256, 4, 16, 256, 256, 3, 2, 16, 0, 256, 16, 256, 16, 256], (1, 4, 5, 10, 12, 14)),
                             (q.coli_moe_combine_grad, [0, 256, 4, 16, 256, 256, 3, 2, 16, 0, 256, 16, 256, 16, 256, 256], (1, 4, 5, 10, 12, 14, 15))):
        for i in places:
            a = list(args)
            a[i] = t
            refused(1, fn, *a, **kw)


# ------------------------------------------------------------------ sort


def plain_sort(ids, E):
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    key = np.where(ok, flat, E)
    order = np.argsort(key, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(len(order))
    live = int(ok.sum())
    return (np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])]), np.where(np.arange(len(order)) < live, order, -1),
            np.where(ok, place, -1), live)


def check_sort(T, K, E, ids, hidden, dtype, ldx=None, ldr=None, off=0, bad=False):
    g = torch.Generator().manual_seed(T * 31 + hidden)
    x = torch.randn(T, hidden, generator=g).to(DT[dtype])
    _, xv = rows_at(x, ldx or hidden, off, dtype)
    rows_flat, rv = rows_at(torch.full((T * K, hidden), -7.0), ldr or hidden, off, dtype)
    before = rows_flat.clone()
    i32 = lambda n: torch.full((n,), -99, dtype=torch.int32, device="cuda")  # noqa: E731
    offsets, perm, place, w = i32(E + 2), i32(T * K + 1), i32(T * K + 1), ws()
    q.coli_moe_sort_rows(E, K, ACT[dtype], xv, T, hidden, xv.stride(0), torch.from_numpy(ids).int().cuda(), offsets, perm, place, rv, rv.stride(0), w)
    assert q.coli_moe_error_word(w) == (q.DEVERR_EXPERT_ID if bad else 0)
    wo, wp, wl, live = plain_sort(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), np.append(wo, -99))
    assert np.array_equal(perm.cpu().numpy(), np.append(wp, -99))
    assert np.array_equal(place.cpu().numpy(), np.append(wl, -99))
    assert torch.equal(rv[:live].cpu(), x[torch.from_numpy(wp[:live] // K)])
    rv[:live] = -7.0                                       # everything else as it was
    assert torch.equal(rows_flat.view(torch.uint8), before.view(torch.uint8))
    # the sort alone gives the same
    o2, p2, l2 = i32(E + 2), i32(T * K + 1), i32(T * K + 1)
    q.coli_moe_sort_rows(E, K, ACT[dtype], None, T, hidden, 0, torch.from_numpy(ids).int().cuda(), o2, p2, l2, None, 0, ws())
    assert torch.equal(o2, offsets) and torch.equal(p2, perm) and torch.equal(l2, place)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,E,hidden", [(1, 1, 1, 1), (1, 8, 256, 6144), (3, 2, 5, 7), (8, 4, 16, 256), (61, 6, 64, 1001), (256, 8, 64, 64),
                                          (257, 8, 64, 96), (700, 3, 1024, 40), (1, 32, 1024, 24), (2049, 1, 1, 16), (3001, 7, 200, 30), (9000, 8, 300, 8),
                                          (641, 4, 8, 6144), (2600, 1, 3, 20008), (2700, 1, 3, 8248), (1300, 2, 16, 2048), (330, 8, 1000, 10240)])
def test_sort(T, K, E, hidden, dtype):
    rng = np.random.default_rng(T + E)
    check_sort(T, K, E, rng.integers(0, E, (T, K)), hidden, dtype)            # (a token may name an expert twice)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 2000])
def test_sort_left_out_slots(T):
    rng = np.random.default_rng(T)
    ids = rng.integers(0, 32, (T, 4))
    check_sort(T, 4, 32, np.where(rng.random((T, 4)) < 0.3, -1, ids), 72, "bf16")
    check_sort(T, 4, 32, np.full((T, 4), -1), 72, "bf16")                     # nothing is left
    check_sort(T, 4, 32, np.where(np.arange(T)[:, None] == T // 2, ids, -1), 72, "f32")
    check_sort(T, 4, 32, np.full((T, 4), 31), 72, "f32")                      # all on one expert
    for worst in (32, -2, 2 ** 31 - 1, -2 ** 31):
        b = ids.copy()
        b[T // 3, 1] = worst
        check_sort(T, 4, 32, b, 72, "bf16", bad=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [30, 1000])
def test_sort_strides(T, dtype):
    ids = np.random.default_rng(5).integers(0, 8, (T, 3))
    for hidden, ldx, ldr, off in ((64, 64, 96, 0), (64, 72, 65, 0), (64, 64, 64, 1), (63, 64, 64, 0), (66, 66, 70, 2), (65, 80, 65, 3)):
        check_sort(T, 3, 8, ids, hidden, dtype, ldx, ldr, off)


@pytest.mark.gpu
def test_sort_of_no_tokens():
    offsets = torch.full((9,), 7, dtype=torch.int32, device="cuda")
    q.coli_moe_sort_rows(8, 2, 0, None, 0, 0, 0, None, offsets, None, None, None, 0, ws())
    assert offsets.tolist() == [0] * 9


# ------------------------------------------------------------------ combine and its gradient


class Batch:
    """Random rows, places (a part of the slots without one, rows that no slot names), weights."""

    def __init__(self, T, K, hidden, act, out, masked=0.2, spare=5, seed=0, ldy=None, ldo=None, off=0):
        rng = np.random.default_rng(seed + T * 7 + K + hidden)
        n = T * K
        self.T, self.K, self.hidden, self.act, self.out = T, K, hidden, act, out
        live = rng.random(n) >= masked
        self.rows = int(live.sum()) + spare
        place = np.full(n, -1)
        place[live] = rng.permutation(self.rows)[:live.sum()]
        self.place = place.reshape(T, K)
        y = torch.from_numpy(rng.standard_normal((self.rows, hidden))).to(DT[act])
        spare_rows = np.setdiff1d(np.arange(self.rows), place)
        y[spare_rows] = float("nan")                          # what no slot names is not read
        self.spare = spare_rows
        self.yflat, self.yv = rows_at(y, ldy or hidden, off, act)
        self.y = np.nan_to_num(y.double().numpy())
        self.w = rng.random((T, K)).astype(np.float32)
        self.add = torch.from_numpy(rng.standard_normal((T, hidden))).to(DT[out])
        self.dout = torch.from_numpy(rng.standard_normal((T, hidden))).to(DT[out])
        self.ldo, self.off = ldo or hidden, off
        self.d_place = torch.from_numpy(self.place).int().cuda()
        self.d_w = torch.from_numpy(self.w).cuda()

    def combine(self, w=True, add=True, in_place=False, stream=None):
        flat, out = rows_at(torch.full((self.T, self.hidden), -7.0), self.ldo, self.off, self.out)
        a = None
        if add:
            a = rows_at(self.add, self.ldo, self.off, self.out)[1]
            if in_place:
                out.copy_(a)
                a = out
        W = ws()
        q.coli_moe_combine(ACT[self.act], self.yv, self.rows, self.yv.stride(0), self.d_place, self.d_w if w else None, self.T, self.K, self.hidden,
                           ACT[self.out], a, self.ldo if add else 0, out, self.ldo, W, stream=stream)
        assert q.coli_moe_error_word(W) == 0
        rest = flat.clone()
        rest[self.off:self.off + self.T * self.ldo].view(self.T, self.ldo)[:, :self.hidden] = float("nan")
        assert torch.isnan(rest).all()
        return out.double().cpu().numpy()

    def want(self, w=True, add=True):
        """The sums and the sums of magnitudes."""
        f = np.where(self.place >= 0, self.w.astype(np.float64) if w else 1.0, 0.0)
        terms = self.y[np.maximum(self.place, 0)] * f[:, :, None]
        s, m = terms.sum(1), np.abs(terms).sum(1)
        if add:
            s, m = s + self.add.double().numpy(), m + np.abs(self.add.double().numpy())
        return s, m

    def check(self, w=True, add=True, **kw):
        got = self.combine(w, add, **kw)
        s, m = self.want(w, add)
        tol = (self.K + 1) * 2.0 ** -24 * m
        if self.out == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(s) + tol)
        assert (np.abs(got - s) <= tol).all()
        return got


SHAPES = [(1, 1, 1), (1, 8, 6144), (7, 3, 8), (4, 32, 264), (61, 6, 1001), (300, 8, 512), (5, 9, 2056), (2, 10, 4100), (700, 5, 1001), (90, 9, 4100),
          (2500, 2, 130), (6000, 1, 77)]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,hidden", SHAPES)
def test_combine(T, K, hidden, act, out):
    b = Batch(T, K, hidden, act, out)
    for w in (True, False):
        for add in (True, False):
            got = b.check(w, add)
            empty = (b.place < 0).all(1)                       # tokens without a row
            assert np.array_equal(got[empty], b.add.double().numpy()[empty] if add else np.zeros_like(got[empty]))
    assert np.array_equal(b.combine(in_place=True), b.combine())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("hidden,ldy,ldo,off", [(64, 72, 80, 0), (64, 65, 64, 0), (64, 64, 64, 1), (63, 64, 64, 0), (68, 68, 76, 4), (72, 72, 74, 2)])
def test_combine_strides(act, hidden, ldy, ldo, off):
    for out in ("f32", "bf16"):
        for T in (37, 6000):
            b = Batch(T, 5 if T == 37 else 2, hidden, act, out, ldy=ldy, ldo=ldo, off=off)
            b.check()
            check_grad(b)


@pytest.mark.gpu
def test_combine_bad_places():
    """Places outside the rows add nothing, are written nowhere and are reported; nothing else changes."""
    b = Batch(20, 4, 64, "bf16", "f32", masked=0.0, spare=0)
    good = b.place.copy()
    for worst in (b.rows, -2, 2 ** 31 - 1, -2 ** 31):
        b.place = good.copy()
        b.place[3, 2] = -1                                     # what the plain form takes it for
        s, m = b.want()
        b.place[3, 2] = worst
        place = torch.from_numpy(b.place).int().cuda()
        out, W = torch.empty(20, 64, device="cuda"), ws()
        q.coli_moe_combine(1, b.yv, b.rows, 64, place, b.d_w, 20, 4, 64, 0, b.add.cuda(), 64, out, 64, W)
        assert q.coli_moe_error_word(W) == q.DEVERR_GROUPING
        assert (np.abs(out.double().cpu().numpy() - s) <= 5 * 2.0 ** -24 * m).all()
        dy, dw, W = torch.full((b.rows, 64), -7.0, dtype=torch.bfloat16, device="cuda"), torch.empty(20, 4, device="cuda"), ws()
        q.coli_moe_combine_grad(1, b.yv, b.rows, 64, place, b.d_w, 20, 4, 64, 0, b.dout.cuda(), 64, dy, 64, dw, W)
        assert q.coli_moe_error_word(W) == q.DEVERR_GROUPING and dw[3, 2] == 0
        left = np.setdiff1d(np.arange(b.rows), b.place)
        assert len(left) == 1 and (dy[left] == -7.0).all() and (dy != -7.0).any(1).sum() == b.rows - 1


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_combine_carries_what_is_not_finite(value):
    """In its own column of the tokens that name the row, a weight of 0 included; nowhere else."""
    b = Batch(9, 3, 40, "f32", "f32", masked=0.0, spare=0)
    b.yv[b.place[4, 1], 7] = value
    b.d_w[4, 1] = 0.0
    got = b.combine()
    assert np.isnan(got[4, 7]) and np.isfinite(np.delete(got.reshape(-1), 4 * 40 + 7)).all()


def threads_of(items):
    pieces = -(-items // 256)
    return -(-(-(-items // pieces)) // 32) * 32


def check_grad(b, use_w=True):
    dyflat, dy = rows_at(torch.full((b.rows, b.hidden), -7.0), b.yv.stride(0), b.off, b.act)
    dw, W = torch.full((b.T, b.K), -7.0, device="cuda"), ws()
    dout = rows_at(b.dout, b.ldo, b.off, b.out)[1]
    args = ACT[b.act], b.yv, b.rows, b.yv.stride(0), b.d_place, b.d_w if use_w else None, b.T, b.K, b.hidden, ACT[b.out], dout, b.ldo
    q.coli_moe_combine_grad(*args, dy, dy.stride(0), dw, W)
    assert q.coli_moe_error_word(W) == 0
    d = b.dout.double().numpy()
    # rows: one product, rounded to float32 and to the type
    live = b.place >= 0
    f = b.w.astype(np.float64) if use_w else np.ones_like(b.w, np.float64)
    want = np.full((b.rows, b.hidden), -7.0)
    want[b.place[live]] = (d[:, None] * f[:, :, None])[live]
    got = dy.double().cpu().numpy()
    assert (np.abs(got - want) <= (2.0 ** -24 + (2.0 ** -8 if b.act == "bf16" else 0)) * 1.01 * np.abs(want) + 2.0 ** -126).all()
    rest = dyflat.clone()
    rest[b.off:b.off + max(b.rows, 1) * dy.stride(0)].view(-1, dy.stride(0))[:b.rows, :b.hidden] = float("nan")
    assert torch.isnan(rest).all()
    # weights: a thread adds its elements one by one, lanes and warps are added in 13 steps at most
    terms = d[:, None] * b.y[np.maximum(b.place, 0)]
    steps = max(-(-b.hidden // v // threads_of(-(-b.hidden // v))) * v for v in (1, 4, 8)) + 8 + 13
    s, m = np.where(live, terms.sum(2), 0.0), np.abs(terms).sum(2)
    assert (np.abs(dw.double().cpu().numpy() - s) <= steps * 2.0 ** -24 * m).all()
    assert (dw.cpu().numpy()[~live] == 0).all()
    # each alone, bit for bit
    dy2, dw2 = torch.full_like(dy, -7.0), torch.full_like(dw, -7.0)
    q.coli_moe_combine_grad(*args, dy2, dy2.stride(0), None, ws())
    q.coli_moe_combine_grad(*args, None, 0, dw2, ws())
    assert torch.equal(dy2, dy) and torch.equal(dw2, dw)
    return dy, dw


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,hidden", SHAPES)
def test_grad(T, K, hidden, act, out):
    b = Batch(T, K, hidden, act, out)
    check_grad(b)
    check_grad(b, use_w=False)


@pytest.mark.gpu
def test_grad_against_differences():
    """The sum is linear in the rows and in the weights: a step in either changes <dout, out> by the gradient times it,
    but for the roundings of the two sums."""
    b = Batch(33, 4, 96, "f32", "f32", spare=0)
    dy, dw = check_grad(b)
    rng = np.random.default_rng(1)
    d = b.dout.double().numpy()
    base, m = b.combine(), b.want()[1]
    slack = 2 * 6 * 2.0 ** -24 * (np.abs(d) * m * 4).sum()
    step = rng.standard_normal(b.w.shape).astype(np.float32)
    w0 = b.d_w.clone()
    b.d_w = w0 + torch.from_numpy(step).cuda()
    moved = (d * (b.combine() - base)).sum()
    exact_step = (b.d_w.double() - w0.double()).cpu().numpy()
    assert abs(moved - (dw.double().cpu().numpy() * exact_step).sum()) <= slack
    b.d_w = w0
    ystep = torch.from_numpy(rng.standard_normal(b.y.shape)).float().cuda()
    y0 = b.yv.clone()
    b.yv.copy_(y0 + ystep)
    moved = (d * (b.combine() - base)).sum()
    exact_step = (b.yv.double() - y0.double()).cpu().numpy()
    assert abs(moved - (dy.double().cpu().numpy() * exact_step).sum()) <= slack
    assert abs(moved) > 100 * slack


@pytest.mark.gpu
@pytest.mark.parametrize("T,hidden", [(50, 136), (1500, 136), (1500, 33)])
def test_sort_and_its_gradient(T, hidden):
    """The rows' gradients combined without weights are the gradient in x: <rows(x), dr> = <x, dx>, exactly the
    transposed copy."""
    rng = np.random.default_rng(T)
    K, E = 4, 16
    ids = rng.integers(0, E, (T, K))
    ids[rng.random((T, K)) < 0.1] = -1
    x = torch.randint(-8, 9, (T, hidden)).float()
    place = torch.empty(T * K, dtype=torch.int32, device="cuda")
    rows = torch.zeros(T * K, hidden, device="cuda")
    W = ws()
    q.coli_moe_sort_rows(E, K, 0, x.cuda(), T, hidden, hidden, torch.from_numpy(ids).int().cuda(), torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                         torch.empty(T * K, dtype=torch.int32, device="cuda"), place, rows, hidden, W)
    dr = torch.randint(-8, 9, (T * K, hidden)).float().cuda()
    dx = torch.empty(T, hidden, device="cuda")
    q.coli_moe_combine(0, dr, T * K, hidden, place, None, T, K, hidden, 0, None, 0, dx, hidden, W)
    assert q.coli_moe_error_word(W) == 0
    live = int((ids >= 0).sum())
    assert (rows[:live].double() * dr[:live].double()).sum() == (x.cuda().double() * dx.double()).sum()   # whole numbers
    want = np.zeros((T, hidden))
    p = place.cpu().numpy().reshape(T, K)
    for k in range(K):
        have = p[:, k] >= 0
        want[have] += dr.cpu().numpy()[p[have, k]]
    assert np.array_equal(dx.cpu().numpy(), want)


@pytest.mark.gpu
def test_training_step_in_a_graph():
    """Sort, weighted sum and both gradients captured, replayed on new inputs, against the direct calls; on a side stream."""
    T, K, E, H = 700, 4, 16, 72
    rng = np.random.default_rng(8)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    x, ids, w = torch.zeros(T, H, device="cuda"), i32(T * K), torch.zeros(T, K, device="cuda")
    dout = torch.zeros(T, H, device="cuda")
    offsets, perm, place = i32(E + 1), i32(T * K), i32(T * K)
    rows, dy = torch.zeros(T * K, H, device="cuda"), torch.zeros(T * K, H, device="cuda")
    out, dx, dw, W = torch.zeros(T, H, device="cuda"), torch.zeros(T, H, device="cuda"), torch.zeros(T, K, device="cuda"), ws()

    def step():
        q.coli_moe_sort_rows(E, K, 0, x, T, H, H, ids, offsets, perm, place, rows, H, W)
        q.coli_moe_combine(0, rows, T * K, H, place, w, T, K, H, 0, x, H, out, H, W)
        q.coli_moe_combine_grad(0, rows, T * K, H, place, w, T, K, H, 0, dout, H, dy, H, dw, W)
        q.coli_moe_combine(0, dy, T * K, H, place, None, T, K, H, 0, dout, H, dx, H, W)

    def inputs():
        x.copy_(torch.from_numpy(rng.standard_normal((T, H))))
        dout.copy_(torch.from_numpy(rng.standard_normal((T, H))))
        w.copy_(torch.from_numpy(rng.random((T, K))))
        ids.copy_(torch.from_numpy(np.where(rng.random(T * K) < 0.1, -1, rng.integers(0, E, T * K))))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        inputs()
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for _ in range(3):
            inputs()
            rows.zero_(), dy.zero_()
            graph.replay()
            got = [t.clone() for t in (offsets, perm, place, rows, out, dy, dw, dx)]
            rows.zero_(), dy.zero_()
            step()
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, (offsets, perm, place, rows, out, dy, dw, dx)))
            # out = x (1 + sum of the placed weights)
            live = (ids.view(T, K) >= 0).double()
            f = 1 + (w.double() * live).sum(1, keepdim=True)
            assert (out.double() - x.double() * f).abs().max() <= 6 * 2.0 ** -24 * 10 * f.max()
    assert q.coli_moe_error_word(W) == 0




@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [1024, 64, 33])
@pytest.mark.parametrize("T", [400, 1200])
def test_chain_of_layers(T, hidden):
    """Every call reads what the one before it has just written, over and over, eagerly and in a graph: x -> rows -> their
    weighted sum with x -> the next x; all terms of a sum have one sign, so that a layer is within its roundings of the value."""
    K, E, L = 4, 24, 6
    rng = np.random.default_rng(T + hidden)
    i32 = lambda v: torch.from_numpy(np.ascontiguousarray(v)).int().cuda()  # noqa: E731
    ids = [np.argsort(rng.random((T, E)), 1)[:, :K] for _ in range(L)]
    w = [np.exp2(rng.integers(-2, 1, (T, K))).astype(np.float32) for _ in range(L)]
    dev_ids, dev_w = [i32(v) for v in ids], [torch.from_numpy(v).cuda() for v in w]
    xs = [torch.zeros(T, hidden, device="cuda") for _ in range(L + 1)]
    rows = torch.zeros(T * K, hidden, device="cuda")
    offsets, perm, place, W = i32(np.zeros(E + 1)), i32(np.zeros(T * K)), i32(np.zeros(T * K)), ws()

    def run():
        for i in range(L):
            q.coli_moe_sort_rows(E, K, 0, xs[i], T, hidden, hidden, dev_ids[i], offsets, perm, place, rows, hidden, W)
            q.coli_moe_combine(0, rows, T * K, hidden, place, dev_w[i], T, K, hidden, 0, xs[i], hidden, xs[i + 1], hidden, W)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
        for call in (run, graph.replay, run, graph.replay):
            x = torch.from_numpy(rng.integers(-3, 4, (T, hidden))).float()
            xs[0].copy_(x)
            call()
            want = x.double().numpy()
            for i in range(L):
                want = want * (1 + w[i].astype(np.float64).sum(1, keepdims=True))
            got = xs[L].double().cpu().numpy()
            assert (np.abs(got - want) <= L * (K + 1) * 2.0 ** -24 * np.abs(want)).all()
    assert q.coli_moe_error_word(W) == 0
