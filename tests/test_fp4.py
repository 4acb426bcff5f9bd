"""Microscaled 4-bit rows: quantisation, its inverse and the product, against plain 64-bit arithmetic.

Quantisation is defined exactly, so its bytes are compared for equality.  The product's sums are
float32: cases whose partial sums all fit 24 bits are compared for equality too, the others with a
bound from the number of additions."""
import numpy as np
import pytest
import torch

import _fp4 as ref

q = pytest.importorskip("quantized_routed_expert_noaux_b200")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACT = {"f32": 0, "bf16": 1}


def ws():
    return torch.zeros(512, dtype=torch.uint8, device="cuda")


def run_quantize(x, fmt, layout=0, index=None, div=1, rows=None, k=None, w=None):
    """x: 2-d device tensor (its row stride is used) -> codes, scales, row scales as numpy."""
    k = x.shape[1] if k is None else k
    rows = x.shape[0] if rows is None else rows
    w = ws() if w is None else w
    act = 0 if x.dtype == torch.float32 else 1
    codes = torch.full((rows, k // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((q.coli_moe_fp4_scale_bytes(fmt, layout, rows, k),), 0xA5, dtype=torch.uint8, device="cuda")
    row = torch.full((rows,), -7.0, device="cuda")
    q.coli_moe_fp4_quantize(fmt, layout, act, x, x.shape[0], x.stride(0), index, div, rows, k, codes, scales, row, w)
    return codes, scales, row, w


def check_quantized(got, x64, fmt, layout, k):
    codes, scales, row, w = got
    code, byte, rs = ref.quantize(x64, fmt)
    want = ref.rows_layout(byte, fmt, k).reshape(-1) if layout == 0 else ref.tiles_layout(byte, fmt, k)
    assert np.array_equal(scales.cpu().numpy(), want)
    assert np.array_equal(row.cpu().numpy(), rs)
    assert np.array_equal(ref.unpack(codes.cpu().numpy()), code)
    assert q.coli_moe_error_word(w) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k,layout", [(1, 32, 0), (1, 6144, 0), (5, 96, 1), (37, 1024, 0), (130, 1056, 1), (257, 256, 1),
                                           (3, 8192, 0), (2, 20000, 0), (129, 2080, 1)])
def test_quantize(fmt, dtype, rows, k, layout):
    g = torch.Generator().manual_seed(rows * 7 + k)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-8, 8, (rows, k // 32, 1), generator=g).float().expand(rows, k // 32, 32)).reshape(rows, k)
    x = x.to(DT[dtype])
    check_quantized(run_quantize(x.cuda(), fmt, layout), x.double().numpy(), fmt, layout, k)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_every_tie(fmt, dtype):
    """Every block scale significand with elements on, just above and just below every midpoint."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for s in range(8, 16):                                # e4m3 significands
        for shift in (-3, 0, 2):
            blocks = []
            for m in mids:
                v = np.full(16, 0.0)
                v[0] = 6.0
                v[1:8], v[8:15] = mids, -mids
                blocks.append(v * s / 8 * 2.0 ** shift)
                w = v.copy()
                eps = 2.0 ** -23 if dtype == "f32" else 2.0 ** -7
                w[1:8] *= 1 + eps
                w[8:15] *= 1 - eps
                blocks.append(w * s / 8 * 2.0 ** shift)
            rows.append(np.concatenate(blocks + [np.zeros(16)] * 2))
    # block maxima on the midpoints of two e4m3 values
    rows.append(np.concatenate([np.r_[6.0 * (17 + 2 * i) / 16 * 2.0 ** (-i % 3), np.zeros(15)] for i in range(16)]))
    x = torch.tensor(np.stack(rows), dtype=torch.float64).to(DT[dtype])
    check_quantized(run_quantize(x.cuda(), fmt), x.double().numpy(), fmt, 0, x.shape[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_extremes(fmt, dtype):
    """Rows of zeros, the smallest and largest finite values, NaN and infinities, negative zeros."""
    x = torch.zeros(12, 64, dtype=torch.float32)
    g = torch.Generator().manual_seed(3)
    x[1] = torch.randn(64, generator=g) * 1e-38
    x[2] = torch.randn(64, generator=g) * 3e-39          # subnormal in both types
    x[3] = 3.3e38 * (torch.rand(64, generator=g) - 0.5)
    x[4] = torch.finfo(DT[dtype]).max
    x[5] = torch.randn(64, generator=g)
    x[5, 17] = float("nan")
    x[6] = torch.randn(64, generator=g)
    x[6, 40] = float("inf")
    x[7] = float("-inf")
    x[8] = -0.0
    x[9, 5] = -2.0 ** -126
    x[10] = torch.randn(64, generator=g)
    x[10, :16] *= 2.0 ** -20                               # a block far below the row's largest
    x[11, 0] = 2.0 ** 127
    x[11, 33] = 1.0
    x = x.to(DT[dtype])
    check_quantized(run_quantize(x.cuda(), fmt), x.double().numpy(), fmt, 0, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_gather_and_strides(fmt):
    g = torch.Generator().manual_seed(9)
    wide = torch.randn(21, 352, generator=g).to(torch.bfloat16)
    x = wide[:, 32:320]                                     # row stride 352, 64 bytes in
    perm = torch.randperm(21 * 4, generator=g).to(torch.int32)
    got = run_quantize(wide.cuda()[:, 32:320], fmt, 0, perm.cuda(), 4, 84)
    check_quantized(got, x[(perm // 4).long()].double().numpy(), fmt, 0, 288)
    # a row may be taken many times or never; bad indices give rows of zeros and an error code
    idx = torch.tensor([5, 5, 20, -1, 0, 21, 5], dtype=torch.int32)
    codes, scales, row, w = run_quantize(wide.cuda()[:, 32:320], fmt, 0, idx.cuda(), 1, 7)
    x64 = x[idx.clamp(0, 20).long()].double().numpy()
    x64[[3, 5]] = 0.0
    code, byte, rs = ref.quantize(x64, fmt)
    assert np.array_equal(ref.unpack(codes.cpu().numpy()), code)
    assert np.array_equal(scales.cpu().numpy(), ref.rows_layout(byte, fmt, 288).reshape(-1))
    assert np.array_equal(row.cpu().numpy(), rs)
    assert q.coli_moe_error_word(w) == q.DEVERR_GROUPING


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,div,k", [(257, 4, 288), (600, 8, 64), (130, 9, 6144), (3, 500, 1056)])
def test_quantize_many_copies(fmt, dtype, T, div, k):
    """Enough rows per source row that each source row is quantised once: as a permutation of the slots; with
    one source row taken by most; with bad indices among them."""
    g = torch.Generator().manual_seed(T + k)
    x = (torch.randn(T, k, generator=g) * 3).to(DT[dtype])
    x[1, 5] = float("nan")
    n = T * div
    for index in (torch.randperm(n, generator=g), torch.where(torch.rand(n, generator=g) < 0.8, div * (T // 2), torch.randint(0, n, (n,), generator=g))):
        index = index.to(torch.int32)
        got = run_quantize(x.cuda(), fmt, 0, index.cuda(), div, n)
        check_quantized(got, x[(index // div).long()].double().numpy(), fmt, 0, k)
    index[[0, n // 2, n - 1]] = torch.tensor([-1, n, -2 ** 31], dtype=torch.int64).to(torch.int32)
    codes, scales, row, w = run_quantize(x.cuda(), fmt, 0, index.cuda(), div, n)
    x64 = x[(index // div).clamp(0, T - 1).long()].double().numpy()
    x64[[0, n // 2, n - 1]] = 0.0
    code, byte, rs = ref.quantize(x64, fmt)
    assert np.array_equal(ref.unpack(codes.cpu().numpy()), code) and np.array_equal(row.cpu().numpy(), rs)
    assert np.array_equal(scales.cpu().numpy(), ref.rows_layout(byte, fmt, k).reshape(-1))
    assert q.coli_moe_error_word(w) == q.DEVERR_GROUPING


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
def test_dequantize(fmt, dtype, layout):
    """Every code under every scale byte; a row scale that is no power of two; rows further apart."""
    rng = np.random.default_rng(4)
    rows, k = 131, 288
    code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    byte = rng.integers(0, 256 if fmt == 0 else 128, (rows, k // ref.BLOCK[fmt])).astype(np.uint8)
    if fmt == 0:
        byte = byte % 200 + 20                              # the products stay finite
        byte[0, 0], byte[1, 1] = 0, 255
    rs = (rng.random(rows) + 0.5).astype(np.float32)
    lay = ref.rows_layout(byte, fmt, k).reshape(-1) if layout == 0 else ref.tiles_layout(byte, fmt, k)
    out = torch.full((rows, 320), -7.0, dtype=DT[dtype], device="cuda")
    q.coli_moe_fp4_dequantize(fmt, layout, torch.from_numpy(ref.pack(code)).cuda(), torch.from_numpy(lay).cuda(),
                              torch.from_numpy(rs).cuda(), rows, k, ACT[dtype], out, 320)
    want = ref.values(code, byte, rs, fmt)
    got = out.double().cpu().numpy()
    assert (got[:, k:] == -7.0).all()
    got = got[:, :k]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fine = ~np.isnan(want)
    # code * block scale is exact, the row scale's product is rounded to float32 once, and to bf16 once
    tol = (2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0)) * 1.01
    assert (np.abs(got - want)[fine] <= tol * np.abs(want)[fine] + 2.0 ** -126).all()


# ------------------------------------------------------------------ product


def random_operand(rng, rows, k, fmt, exact):
    """codes, scale bytes, row scales; `exact`: few scales, all powers of two near 1."""
    code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    nb = k // ref.BLOCK[fmt]
    if exact:
        byte = (rng.integers(127, 129, (rows, nb)) if fmt == 0 else rng.choice(np.array([0x38, 0x40]), (rows, nb))).astype(np.uint8)
        row = np.ldexp(1.0, rng.integers(-3, 4, rows)).astype(np.float32)
    else:
        byte = (rng.integers(117, 130, (rows, nb)) if fmt == 0 else rng.integers(0, 127, (rows, nb))).astype(np.uint8)
        row = (rng.random(rows) + 0.5).astype(np.float32)
    return code, byte, row


class Product:
    """Operands of one product on the host and the device."""

    def __init__(self, fmt, sizes, n, k, exact, seed=0, tail=0, row_scales=True):
        rng = np.random.default_rng(seed + 31 * n + k)
        self.fmt, self.n, self.k, self.sizes = fmt, n, k, sizes
        self.rows = sum(sizes) + tail
        self.a = random_operand(rng, self.rows, k, fmt, exact)
        self.w = [random_operand(rng, n, k, fmt, exact) for _ in sizes]
        if not row_scales:
            self.a = (*self.a[:2], None)
            self.w = [(*w[:2], None) for w in self.w]
        self.offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
        self.dev = [dev(ref.pack(self.a[0])), dev(ref.rows_layout(self.a[1], fmt, k)), dev(self.a[2]) if row_scales else None,
                    dev(np.stack([ref.pack(w[0]) for w in self.w])), dev(np.stack([ref.tiles_layout(w[1], fmt, k) for w in self.w])),
                    dev(np.stack([w[2] for w in self.w])) if row_scales else None]
        self.dev_offsets = dev(self.offsets)

    def call(self, out, act, grouped=True, offsets=None, w=None):
        c = self.dev
        w = ws() if w is None else w
        off = (self.dev_offsets if offsets is None else offsets) if grouped else None
        q.coli_moe_fp4_product(self.fmt, q.fp4_rows_for(*c[:3]), q.fp4_mats_for(*c[3:]), self.k, off, act, out, out.stride(0), w)
        return w

    def want(self):
        """float64 results and, per element, the largest partial sum over runs of 64 elements."""
        y = np.zeros((self.rows, self.n))
        big = np.zeros((self.rows, self.n))
        xa = ref.values(*self.a[:2], None, self.fmt)
        for e, w in enumerate(self.w):
            lo, hi = self.offsets[e], self.offsets[e + 1]
            wv = ref.values(*w[:2], None, self.fmt)
            s = np.zeros((hi - lo, self.n))
            b = np.zeros_like(s)
            for j in range(0, self.k, 64):
                s = s + xa[lo:hi, j:j + 64] @ wv[:, j:j + 64].T
                b = np.maximum(b, np.abs(s))
            # the largest single product takes part in the alignment of a step's terms
            b = np.maximum(b, np.abs(xa[lo:hi]).max(1, initial=0)[:, None] * np.abs(wv).max(1)[None, :])
            r = (1.0 if self.a[2] is None else self.a[2][lo:hi].astype(np.float64))
            r = np.multiply.outer(np.broadcast_to(r, hi - lo), np.ones(self.n)) * (1.0 if w[2] is None else w[2].astype(np.float64)[None, :])
            y[lo:hi], big[lo:hi] = s * r, b * np.abs(r)
        return y, big


SHAPES = [  # rows of every group, n, k
    ([1], 128, 256), ([1], 1, 32), ([3], 200, 96), ([16], 64, 64), ([17], 129, 288), ([128], 256, 512), ([129], 130, 1056),
    ([300], 384, 320), ([0, 1, 0, 5, 33, 0], 192, 224), ([7, 0, 140, 1], 136, 544), ([1] * 9, 256, 1024), ([0, 0, 2], 16, 2048),
    ([40, 260], 640, 128), ([1], 384, 6144), ([600], 100, 6144), ([32], 2048, 2048), ([2, 0, 9, 20], 4096, 1024),
    ([int(e % 97 == 3) for e in range(1023)] + [2], 48, 64), ([e % 5 for e in range(1000)], 24, 32), ([0] * 31 + [40] + [0] * 32 + [1], 160, 96),
    ([0] * 9 + [300], 200, 320), ([1] * 20 + [260], 130, 1056),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_product_exact_sums(fmt, i):
    """Codes of every value under scales 1 and 2: terms are multiples of 1/4 and at most 144, so sums of
    6144 terms have at most 2 + 7.2 + 12.6 < 24 bits, and the row scales are powers of two: float32
    results equal the real ones, bf16 results the real ones rounded."""
    sizes, n, k = SHAPES[i]
    p = Product(fmt, sizes, n, k, exact=True)
    y, _ = p.want()
    out = torch.full((p.rows, n + 3), -7.0, device="cuda")
    w = p.call(out, 0)
    assert q.coli_moe_error_word(w) == 0
    assert np.array_equal(out[:, :n].cpu().numpy().astype(np.float64), y)
    assert (out[:, n:] == -7.0).all()
    out = torch.full((p.rows, n), -7.0, dtype=torch.bfloat16, device="cuda")
    p.call(out, 1)
    assert torch.equal(out.cpu(), torch.from_numpy(y).to(torch.float32).to(torch.bfloat16))
    if len(sizes) == 1:  # one matrix: no offsets needed
        dense = torch.full((p.rows, n), -7.0, device="cuda")
        p.call(dense, 0, grouped=False)
        assert np.array_equal(dense.cpu().numpy().astype(np.float64), y)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("row_scales", [True, False])
@pytest.mark.parametrize("sizes,n,k", [([1], 256, 6144), ([33, 0, 150], 200, 1056), ([2, 3], 130, 96)])
def test_product_any_scales(fmt, row_scales, sizes, n, k):
    """Scales of every size.  A term or partial sum is kept to a unit of 2^-23 of the largest
    partial sum (terms of a step are aligned to it and may be cut): at most one such unit for each of
    the k terms; then two roundings by the row scales, and one to bf16."""
    p = Product(fmt, sizes, n, k, exact=False, row_scales=row_scales)
    y, big = p.want()
    for act, out_step in ((0, 0.0), (1, 2.0 ** -8)):
        out = torch.empty(p.rows, n, dtype=torch.float32 if act == 0 else torch.bfloat16, device="cuda")
        p.call(out, act)
        tol = k * 2.0 ** -23 * big + (2 * 2.0 ** -24 + out_step) * 1.01 * (np.abs(y) + k * 2.0 ** -23 * big)
        assert (np.abs(out.double().cpu().numpy() - y) <= tol).all()


@pytest.mark.gpu
def test_product_leaves_other_rows():
    """Rows behind the last group, and rows of groups whose offsets are not ascending, are not written."""
    p = Product(1, [5, 20, 3], 72, 96, exact=True, tail=9)
    y, _ = p.want()
    out = torch.full((p.rows, 72), -7.0, device="cuda")
    w = p.call(out, 0)
    assert q.coli_moe_error_word(w) == 0
    assert np.array_equal(out[:28].cpu().numpy().astype(np.float64), y[:28]) and (out[28:] == -7.0).all()
    for bad in ([0, 5, 3, 28], [0, 5, 25, 1000], [-1, 5, 25, 28]):
        out = torch.full((p.rows, 72), -7.0, device="cuda")
        w = p.call(out, 0, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert q.coli_moe_error_word(w) == q.DEVERR_GROUPING
        assert (out[28:] == -7.0).all() or bad[3] == 28
        if bad[1] == 5 and bad[0] == 0:
            assert np.array_equal(out[:3].cpu().numpy().astype(np.float64), y[:3])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
def test_product_of_quantized_nan(fmt):
    """A NaN in a row reaches that row's results and no other's; a NaN weight its column's."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(5, 256, generator=g)
    x[2, 77] = float("nan")
    w = torch.randn(1, 130, 256, generator=g)
    w[0, 129, 3] = float("inf")
    codes, scales, row, _ = run_quantize(x.cuda(), fmt)
    wc, wsc, wr, _ = run_quantize(w[0].cuda(), fmt, layout=1)
    out = torch.empty(5, 130, device="cuda")
    q.coli_moe_fp4_product(fmt, q.fp4_rows_for(codes, scales, row), q.fp4_mats_for(wc[None], wsc[None], wr[None]), 256, None, 0, out, 130, ws())
    nan = torch.isnan(out.cpu())
    want = torch.zeros(5, 130, dtype=torch.bool)
    want[2], want[:, 129] = True, True
    assert torch.equal(nan, want)


@pytest.mark.gpu
def test_linear_layer_of_three_calls():
    """Quantise weights and activations, multiply, on a stream of its own and from a CUDA graph."""
    g = torch.Generator().manual_seed(11)
    x, w = torch.randn(40, 512, generator=g), torch.randn(300, 512, generator=g) * 0.05
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        xd, wd = x.cuda(), w.cuda()
        wc, wsc, wr, _ = run_quantize(wd, 1, layout=1)
        out = torch.zeros(40, 300, device="cuda")
        codes = torch.empty(40, 256, dtype=torch.uint8, device="cuda")
        scales = torch.empty(40, q.coli_moe_fp4_scale_pitch(1, 512), dtype=torch.uint8, device="cuda")
        row = torch.empty(40, device="cuda")
        W = ws()

        def step():
            q.coli_moe_fp4_quantize(1, 0, 0, xd, 40, 512, None, 1, 40, 512, codes, scales, row, W)
            q.coli_moe_fp4_product(1, q.fp4_rows_for(codes, scales, row), q.fp4_mats_for(wc[None], wsc[None], wr[None]), 512, None, 0, out, 300, W)

        step()
    st.synchronize()
    first = out.cpu()
    xq = ref.values(*ref.quantize(x.numpy(), 1), 1)
    wq = ref.values(*ref.quantize(w.numpy(), 1), 1)
    y = xq @ wq.T
    # 512 terms, each partial sum at most sum |x w|
    assert (np.abs(first.double().numpy() - y) <= 512 * 2.0 ** -23 * (np.abs(xq) @ np.abs(wq).T)).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    x2 = torch.randn(40, 512, generator=g)
    xd.copy_(x2)
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    xq = ref.values(*ref.quantize(x2.numpy(), 1), 1)
    assert (np.abs(out.double().cpu().numpy() - xq @ wq.T) <= 512 * 2.0 ** -23 * (np.abs(xq) @ np.abs(wq).T)).all()
    assert q.coli_moe_error_word(W) == 0


# ------------------------------------------------------------------ refusals (host only)


def refused(status, fn, *args):
    with pytest.raises(q.ColiError) as ei:
        fn(*args, stream=0)
    assert ei.value.status == status


def test_sizes_on_the_host():
    assert q.coli_moe_fp4_scale_pitch(0, 32) == 8 and q.coli_moe_fp4_scale_pitch(1, 288) == 32
    assert q.coli_moe_fp4_scale_bytes(1, 1, 129, 256) == 256 * 16 and q.coli_moe_fp4_scale_bytes(0, 0, 3, 6144) == 3 * 192
    for bad, status in (((2, 32), 1), ((0, 16), 2), ((0, 0), 2), ((1, 2 << 20), 4)):
        with pytest.raises(q.ColiError) as ei:
            q.coli_moe_fp4_scale_pitch(*bad)
        assert ei.value.status == status


def test_quantize_refusals():
    good = [0, 0, 1, 256, 4, 64, None, 1, 4, 64, 512, 1024, 2048, 4096]

    def with_(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return a
    f = q.coli_moe_fp4_quantize
    refused(1, f, *with_(_0=5))
    refused(1, f, *with_(_1=2))
    refused(1, f, *with_(_2=2))
    refused(1, f, *with_(_3=None))
    refused(1, f, *with_(_12=None))
    refused(2, f, *with_(_5=32))            # rows closer than they are long
    refused(2, f, *with_(_9=48, _5=48))     # k
    refused(2, f, *with_(_8=5))             # no index: rows == src_rows
    refused(2, f, *with_(_7=2))
    refused(2, f, *with_(_6=128, _7=0))
    refused(2, f, *with_(_8=-1))
    refused(3, f, *with_(_3=264))
    refused(3, f, *with_(_5=68))            # 136 bytes
    refused(3, f, *with_(_10=516))
    refused(7, f, *with_(_13=None))
    refused(7, f, *with_(_13=4100))
    f(*with_(_8=0, _4=0, _3=None), stream=0)  # no rows: a no-op


def test_dequantize_refusals():
    good = [0, 0, 256, 512, None, 4, 64, 0, 1024, 64]

    def with_(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return a
    f = q.coli_moe_fp4_dequantize
    refused(1, f, *with_(_0=-1))
    refused(1, f, *with_(_7=3))
    refused(1, f, *with_(_3=None))
    refused(2, f, *with_(_9=63))
    refused(2, f, *with_(_6=40))
    refused(3, f, *with_(_9=66))
    refused(3, f, *with_(_8=1032))
    f(*with_(_5=0, _8=None), stream=0)


def test_product_refusals():
    A = lambda **kw: q.FP4Rows(**{**dict(codes=256, scales=512, row_scale=None, rows=4), **kw})  # noqa: E731
    W = lambda **kw: q.FP4Mats(**{**dict(codes=1024, scales=2048, row_scale=None, count=2, n=64, codes_stride=64 * 32,  # noqa: E731
                                         scales_stride=128 * 16, row_scale_stride=0), **kw})
    f = q.coli_moe_fp4_product

    def call(a=None, w=None, fmt=1, k=64, off=4096, act=0, out=8192, ldo=64, wsp=16384):
        return (fmt, a or A(), w or W(), k, off, act, out, ldo, wsp)
    refused(1, f, *call(fmt=3))
    refused(1, f, *call(act=2))
    refused(1, f, *call(a=A(codes=None)))
    refused(1, f, *call(w=W(scales=None)))
    refused(1, f, *call(out=None))
    refused(2, f, *call(k=40))
    refused(2, f, *call(ldo=63))
    refused(2, f, *call(off=None))              # two matrices need offsets
    refused(2, f, *call(w=W(n=0)))
    refused(2, f, *call(w=W(codes_stride=64)))
    refused(2, f, *call(w=W(scales_stride=1024)))
    refused(2, f, *call(w=W(row_scale=64, row_scale_stride=63)))
    refused(3, f, *call(a=A(codes=264)))
    refused(3, f, *call(w=W(codes_stride=64 * 32 + 8)))
    refused(3, f, *call(out=8194))
    refused(3, f, *call(off=4098))
    refused(4, f, *call(w=W(count=1025, codes_stride=64 * 32)))
    refused(4, f, *call(a=A(rows=1 << 30), w=W(n=6144, codes_stride=6144 * 32, scales_stride=6144 * 16), ldo=6144))
    refused(7, f, *call(wsp=None))
    f(*call(a=A(rows=0, codes=None)), stream=0)


# ------------------------------------------------------------------ the calls a user may make beside these


@pytest.mark.gpu
def test_far_apart():
    """Matrices, rows of x and rows of out that lie more than 2^32 bytes apart."""
    fmt, n, k, far = 1, 72, 96, 5 << 30
    p = Product(fmt, [2, 1], n, k, exact=True)
    codes = torch.empty(far + n * k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(far + 128 * ref.pitch(fmt, k), dtype=torch.uint8, device="cuda")
    for e in range(2):
        codes[e * far:][:n * k // 2] = p.dev[3][e].reshape(-1)
        scales[e * far:][:128 * ref.pitch(fmt, k)] = p.dev[4][e]
    w = q.FP4Mats(codes.data_ptr(), scales.data_ptr(), p.dev[5].data_ptr(), 2, n, far, far, n)
    ldo = (1 << 30) + 12
    out = torch.empty(2 * ldo + n, device="cuda")
    q.coli_moe_fp4_product(fmt, q.fp4_rows_for(*p.dev[:3]), w, k, p.dev_offsets, 0, out, ldo, ws())
    y, _ = p.want()
    for i in range(3):
        assert np.array_equal(out[i * ldo:][:n].cpu().numpy().astype(np.float64), y[i])
    del out, codes, scales
    ldx = (1 << 31) + 32
    x = torch.empty(2 * ldx + 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(3, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for i in range(3):
        x[i * ldx:][:64] = rows[i].cuda()
    codes, scales, row = torch.empty(3, 32, dtype=torch.uint8, device="cuda"), torch.empty(3, 16, dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")
    w = ws()
    q.coli_moe_fp4_quantize(1, 0, 1, x, 3, ldx, None, 1, 3, 64, codes, scales, row, w)
    check_quantized((codes, scales.reshape(-1), row, w), rows.double().numpy(), 1, 0, 64)
    q.coli_moe_fp4_dequantize(1, 0, codes, scales, row, 3, 64, 1, x, ldx)
    code, byte, rs = ref.quantize(rows.double().numpy(), 1)
    for i in range(3):  # at most 6 bits: exact in bf16
        assert np.array_equal(x[i * ldx:][:64].double().cpu().numpy(), ref.values(code, byte, rs, 1)[i])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
def test_two_streams_at_once(fmt):
    """Products of different sizes on two streams, the weights shared, each with its own workspace and output."""
    big, small = Product(fmt, [300, 0, 200], 512, 1024, exact=True), Product(fmt, [3], 512, 1024, exact=True, seed=7)
    want = [p.want()[0] for p in (big, small)]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.zeros(p.rows, 512, device="cuda") for _ in range(8)] for p in (big, small)]
    wss = [ws(), ws()]
    torch.cuda.synchronize()
    for i in range(8):
        for j, p in enumerate((big, small)):
            with torch.cuda.stream(st[j]):
                p.call(outs[j][i], 0, w=wss[j])
    torch.cuda.synchronize()
    for j in range(2):
        for o in outs[j]:
            assert np.array_equal(o.cpu().numpy().astype(np.float64), want[j])
        assert q.coli_moe_error_word(wss[j]) == 0


@pytest.mark.gpu
def test_chained_on_one_stream():
    """Kernels that are set up while the one before still runs see what it wrote: quantise, multiply, quantise
    the result, multiply, many times over the same buffers, against the same steps one by one."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 512, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(512, 512, generator=g) * 512 ** -0.5).to(torch.bfloat16).cuda()
    wc, wsc, wr, _ = run_quantize(w, 1, layout=1)
    mats = q.fp4_mats_for(wc[None], wsc[None], wr[None])

    def chain(wait):
        y = x.clone()
        codes, scales, row = torch.empty(40, 256, dtype=torch.uint8, device="cuda"), torch.empty(40, 32, dtype=torch.uint8, device="cuda"), torch.empty(40, device="cuda")
        rows = q.fp4_rows_for(codes, scales, row)
        W = ws()
        for _ in range(30):
            q.coli_moe_fp4_quantize(1, 0, 1, y, 40, 512, None, 1, 40, 512, codes, scales, row, W)
            wait()
            q.coli_moe_fp4_product(1, rows, mats, 512, None, 1, y, 512, W)
            wait()
        torch.cuda.synchronize()
        return y.cpu()
    one = chain(torch.cuda.synchronize)
    assert torch.isfinite(one.float()).all() and one.float().abs().max() > 0
    for _ in range(5):
        assert torch.equal(chain(lambda: None), one)


def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros(1, 64)
    with pytest.raises(q.ColiError) as ei:
        q.coli_moe_fp4_quantize(1, 0, 0, x, 1, 64, None, 1, 1, 64, x, x, x, 256)
    assert ei.value.status == 1
