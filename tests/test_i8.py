"""8-bit rows and their products against plain exact arithmetic.

Quantisation is defined exactly, so codes and scales are compared for equality (SwiGLU's values are float32 results: theirs
by a bound).  The product's sums are whole numbers: where they fit 24 bits and the scales are powers of two, results
are compared for equality too, else with the three roundings to float32 (2^-24 each) and the one to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import synth

q = pytest.importorskip("quantized_routed_expert_noaux_b200")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACT = {"f32": 0, "bf16": 1}
TINY = 127.0 * 2.0 ** -126


def ws():
    return torch.zeros(512, dtype=torch.uint8, device="cuda")


def refused(status, fn, *args, **kw):
    with pytest.raises(q.ColiError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status


def up16(k):
    return -(-k // 16) * 16


# ------------------------------------------------------------------ refusals (host)


def test_refusals():
    Q = [0, 0, 256, 4, 64, 48, 256, 2, 8, 256, 48, 256, 256]

    def quant(status, **kw):
        names = ["act", "swiglu", "x", "src_rows", "ldx", "k", "place", "copies", "rows", "codes", "ldc", "scale", "ws"]
        refused(status, q.coli_moe_i8_quantize, *[kw.get(n, v) for n, v in zip(names, Q)], stream=0)
    quant(1, act=2)
    quant(1, swiglu=2)
    quant(1, x=None)
    quant(1, codes=None)
    quant(1, scale=None)
    quant(2, src_rows=-1)
    quant(2, rows=-1)
    quant(2, k=0)
    quant(2, ldx=47)
    quant(2, swiglu=1)                   # gate and up need 96
    quant(2, ldc=32)
    quant(2, copies=0)
    quant(2, place=None)                 # two copies to nowhere
    quant(2, place=None, copies=1)       # 4 rows to 8
    quant(4, k=131072, ldx=1 << 18, ldc=1 << 18)
    quant(4, rows=(1 << 30) + 1)
    quant(4, src_rows=(1 << 29) + 1)
    quant(3, x=258)
    quant(3, codes=264)
    quant(3, ldc=56)
    quant(3, place=258)
    quant(3, scale=258)
    quant(7, ws=None)
    quant(7, ws=32)

    def product(status, a=(256, 256, 4, 64), w=(256, 256, 2, 8, 64, 512, 8), k=64, offsets=256, out_type=0, out=256, ldo=8, W=256):
        refused(status, q.coli_moe_i8_product, q.I8Rows(*a), q.I8Mats(*w), k, offsets, out_type, out, ldo, W, stream=0)
    product(1, out_type=2)
    product(1, a=(None, 256, 4, 64))
    product(1, w=(None, 256, 2, 8, 64, 512, 8))
    product(1, out=None)
    product(2, a=(256, 256, -1, 64))
    product(2, a=(256, 256, 4, 48))
    product(2, w=(256, 256, 2, 8, 48, 512, 8))
    product(2, w=(256, 256, 0, 8, 64, 512, 8))
    product(2, w=(256, 256, 2, 0, 64, 512, 8))
    product(2, w=(256, 256, 2, 8, 64, 496, 8))
    product(2, w=(256, 256, 2, 8, 64, 512, 7))
    product(2, offsets=None)
    product(2, ldo=7)
    product(2, k=0)
    product(4, w=(256, 256, 1025, 8, 64, 512, 8))
    product(4, k=131072, a=(256, 256, 4, 1 << 18), w=(256, 256, 2, 8, 1 << 18, 1 << 22, 8))
    product(4, a=(256, 256, 4, 1 << 30))
    product(4, a=(256, 256, 1 << 30, 64), w=(256, 256, 64, 4096, 64, 1 << 18, 4096), ldo=4096)
    product(3, a=(264, 256, 4, 64))
    product(3, a=(256, 256, 4, 72))
    product(3, a=(256, 258, 4, 64))
    product(3, w=(256, 256, 2, 8, 64, 520, 8))
    product(3, w=(256, 256, 2, 8, 72, 576, 8))
    product(3, out=258)
    product(3, offsets=257)
    product(7, W=None)
    product(7, W=64)


def test_documented_bounds_are_refused():
    """Each bound that the header gives, one beyond it; all of them end before a launch."""
    big = 1 << 30

    def quant(**kw):
        a = dict(act=0, swiglu=0, x=256, src_rows=4, ldx=64, k=48, place=256, copies=2, rows=8, codes=256, ldc=48, scale=256, ws=256)
        refused(4, q.coli_moe_i8_quantize, *{**a, **kw}.values(), stream=0)
    quant(rows=big + 1)
    quant(src_rows=big + 1, copies=1)
    quant(src_rows=big + 1, copies=1, rows=big + 1, place=None)
    quant(src_rows=big // 2 + 1)
    quant(src_rows=1, copies=big + 1)
    quant(k=131072, ldx=131072, ldc=131072)

    def product(k=64, ldo=8, offsets=256, **kw):
        a = dict(acodes=256, ascale=256, rows=4, ald=64, wcodes=256, wscale=256, count=2, n=8, wld=64, codes_stride=512, scale_stride=8)
        v = list({**a, **kw}.values())
        refused(4, q.coli_moe_i8_product, q.I8Rows(*v[:4]), q.I8Mats(*v[4:]), k, offsets, 0, 256, ldo, 256, stream=0)
    product(k=131072, ald=131072, wld=131072, codes_stride=1 << 21)
    product(rows=big + 1)
    product(ald=big)
    product(wld=big, codes_stride=1 << 34)
    product(codes_stride=1 << 40)
    product(n=1 << 20, wld=1 << 20, codes_stride=(1 << 40) - 16, ldo=1 << 20, scale_stride=1 << 20)   # n * ld = 2^40
    product(n=1 << 20, wld=1 << 20, count=1, offsets=None, ldo=1 << 20)
    product(count=1025)
    # (rows / 16 + 1) * ceil(n / 128) * (count + 1) = 2^31: 2^20 * 2^10 * 2
    product(rows=((1 << 20) - 1) * 16, n=1 << 17, count=1, offsets=None, ldo=1 << 17)


@pytest.mark.parametrize("explicit", [False, True])
def test_any_tensor_off_the_gpu_is_refused(explicit):
    if torch.cuda.is_available():
        pytest.skip("host check: where it runs nothing could be launched on such a pointer")
    kw = {"stream": 0} if explicit else {}
    t = torch.zeros(64)
    a, w = q.I8Rows(256, 256, 4, 64), q.I8Mats(256, 256, 2, 8, 64, 512, 8)
    for fn, args, places in ((q.coli_moe_i8_quantize, [0, 0, 256, 4, 64, 48, 256, 2, 8, 256, 48, 256, 256], (2, 6, 9, 11, 12)),
                             (q.coli_moe_i8_product, [a, w, 64, 256, 0, 256, 8, 256], (3, 5, 7))):
        for i in places:
            args_ = list(args)
            args_[i] = t
            refused(1, fn, *args_, **kw)
    a.device, w.device = 0, 1
    refused(1, q.coli_moe_i8_product, a, w, 64, 256, 0, 256, 8, 256, stream=0)


def test_helpers_refuse_tensors_that_do_not_fit():
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8)  # noqa: E731
    refused(2, q.i8_rows_for, i8(64, 4).t())
    refused(2, q.i8_rows_for, i8(4, 64), torch.zeros(8)[::2])
    refused(2, q.i8_mats_for, i8(2, 64, 8).transpose(1, 2))
    refused(2, q.i8_mats_for, i8(2, 8, 64), torch.zeros(2, 16)[:, ::2])
    refused(1, q.i8_rows_for, i8(4, 64), torch.zeros(4))  # not on a GPU
    refused(1, q.i8_mats_for, i8(2, 8, 64), torch.zeros(2, 8))


def test_helpers_refuse_other_types_and_shapes():
    """Codes that are not int8, scales that are not float32 or not one to a row: the kernels would read others as these, and
    short ones behind their end."""
    i8, f32 = (lambda *s: torch.zeros(*s, dtype=torch.int8)), torch.zeros
    for t in (torch.uint8, torch.int16, torch.float32, torch.bool, torch.float8_e4m3fn):
        refused(1, q.i8_rows_for, torch.zeros(4, 64).to(t), f32(4))
        refused(1, q.i8_mats_for, torch.zeros(2, 8, 64).to(t), f32(2, 8))
    for t in (torch.bfloat16, torch.float64, torch.int32):
        refused(1, q.i8_rows_for, i8(4, 64), f32(4).to(t))
        refused(1, q.i8_mats_for, i8(2, 8, 64), f32(2, 8).to(t))
    for s in ((3,), (5,), (1,), (0,), (4, 1), (1, 4), ()):
        refused(2, q.i8_rows_for, i8(4, 64), f32(s))
    for s in ((1, 8), (2, 1), (2, 7), (2, 9), (3, 8), (16,), (8,), (2, 8, 1), ()):
        refused(2, q.i8_mats_for, i8(2, 8, 64), f32(s))
    for s in ((64,), (1, 4, 64), ()):
        refused(2, q.i8_rows_for, i8(s))
    for s in ((8, 64), (64,), (1, 2, 8, 64)):
        refused(2, q.i8_mats_for, i8(s))


@pytest.mark.gpu
def test_helpers_refuse_other_types_on_the_gpu():
    """The same of types where tensors are on the GPU (a host tensor is refused with the same status)."""
    i8, f32 = (lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")), (lambda *s: torch.zeros(*s, device="cuda"))
    for t in (torch.uint8, torch.int16, torch.float32, torch.bool, torch.float8_e4m3fn):
        refused(1, q.i8_rows_for, f32(4, 64).to(t), f32(4))
        refused(1, q.i8_mats_for, f32(2, 8, 64).to(t), f32(2, 8))
    for t in (torch.bfloat16, torch.float64, torch.int32):
        refused(1, q.i8_rows_for, i8(4, 64), f32(4).to(t))
        refused(1, q.i8_mats_for, i8(2, 8, 64), f32(2, 8).to(t))
    assert q.i8_rows_for(i8(4, 64), f32(4)).rows == 4 and q.i8_mats_for(i8(2, 8, 64), f32(2, 16)[:, :8]).scale_stride == 16


# ------------------------------------------------------------------ quantisation


def plain_quantize(x):
    """Codes and float32 scales of float64 rows (finite, at most float32's 24 bits), exactly."""
    x = np.asarray(x, np.float64)
    m = np.maximum(np.abs(x).max(1, keepdims=True, initial=0.0), TINY)
    a = np.abs(x) * 127                      # 31 bits
    c = np.floor(a / m)
    half = (c + 0.5) * m                     # 32 bits
    c = c + ((a > half) | ((a == half) & (c % 2 == 1)))
    return (np.copysign(c, x)).astype(np.int8), (m[:, 0] / 127).astype(np.float32)


def run_quantize(x, k=None, swiglu=0, place=None, copies=1, rows=None, ldc=None, fill=-99):
    k = x.shape[1] if k is None else k
    rows = x.shape[0] if rows is None else rows
    ldc = up16(k) if ldc is None else ldc
    codes = torch.full((rows, ldc), fill, dtype=torch.int8, device="cuda")
    scale = torch.full((rows,), -7.0, device="cuda")
    w = ws()
    q.coli_moe_i8_quantize(ACT["f32" if x.dtype == torch.float32 else "bf16"], swiglu, x, x.shape[0], x.stride(0), k, place, copies, rows, codes, ldc,
                           scale, w)
    return codes.cpu().numpy(), scale.cpu().numpy(), q.coli_moe_error_word(w)


def check_quantize(x, **kw):
    codes, scale, err = run_quantize(x, **kw)
    k = x.shape[1]
    wc, wsc = plain_quantize(x.double().cpu().numpy())
    assert err == 0
    assert np.array_equal(codes[:, :k], wc)
    assert np.array_equal(scale, wsc)
    assert (codes[:, k:up16(k)] == 0).all() and (codes[:, up16(k):] == -99).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 6144), (3, 15), (5, 16), (9, 17), (37, 1001), (130, 2048), (131, 2064), (3, 8192), (2, 20000), (5, 2047),
                                    (3, 12301), (2, 20001), (1100, 2304), (1030, 1040), (1500, 6144), (1024, 12288), (1200, 1001), (1025, 3001)])
def test_quantize(rows, k, dtype):
    g = torch.Generator().manual_seed(rows + k)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g).float())
    check_quantize(x.to(DT[dtype]).cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_every_tie(dtype):
    """Rows whose maximum makes halves representable, with elements on, just below and just above each of them; and
    maxima of all significands with elements of half the maximum (63.5)."""
    rows = []
    for e in (-100, -3, 0, 60):
        half = (np.arange(127) + 0.5)
        eps = 2.0 ** -23 if dtype == "f32" else 2.0 ** -7
        for v in (half, half * (1 + eps), half * (1 - eps), -half):
            rows.append(np.concatenate([[127.0], v]) * 2.0 ** e)
    rng = np.random.default_rng(2)
    bits = 23 if dtype == "f32" else 7
    for i in range(128):
        m = 1 + (rng.integers(0, 1 << bits) if dtype == "f32" else i) / (1 << bits)
        rows.append(np.concatenate([[m], m * 2.0 ** -np.arange(1, 9), -m * 2.0 ** -np.arange(1, 9.0),
                                    m / 2 * (1 + np.array([1, -1, 2, -2]) * 2.0 ** -bits), np.zeros(107)]))
    x = torch.tensor(np.stack(rows)).to(DT[dtype])
    check_quantize(x.cuda())


@pytest.mark.gpu
def test_quantize_near_ties():
    """float32 elements next to a half of the real quotient, closer than float32 arithmetic tells apart."""
    rng = np.random.default_rng(3)
    m = (1 + rng.random((400, 1))).astype(np.float32)
    c = rng.integers(0, 127, (400, 63)) + 0.5
    x = (c * m.astype(np.float64) / 127).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-2, 3, x.shape)).astype(np.int32).view(np.float32)
    x = x * rng.choice([-1, 1], x.shape).astype(np.float32)
    x = np.concatenate([m, np.clip(x, -m, m)], 1)
    check_quantize(torch.from_numpy(x).cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_extremes(dtype):
    t = DT[dtype]
    g = torch.Generator().manual_seed(5)
    x = torch.zeros(11, 70)
    x[1] = torch.randn(70, generator=g) * 1e-38
    x[2] = torch.randn(70, generator=g) * 1e-40          # subnormal
    x[3] = torch.randn(70, generator=g) * 1e-36          # about the smallest scale
    x[4] = torch.finfo(t).max
    x[5] = torch.randn(70, generator=g).clamp(-2, 2) * 1.5e38
    x[6] = -0.0
    x[7, 3] = TINY
    x[8, 69] = 2.0 ** -133                               # bf16's smallest
    x[9] = torch.randn(70, generator=g)
    x[9, :35] *= 1e-3
    x[10] = -torch.finfo(t).max
    check_quantize(x.to(t).cuda())
    # rows that are not finite: scale NaN, codes 0; their neighbours as they are
    y = torch.randn(5, 70, generator=g).to(t)
    y[1, 69] = float("nan")
    y[2, 0] = float("inf")
    y[4, 33] = float("-inf")
    codes, scale, err = run_quantize(y.cuda())
    wc, wsc = plain_quantize(torch.nan_to_num(y, 0, 0, 0).double().numpy())
    bad = [1, 2, 4]
    assert err == 0 and np.isnan(scale[bad]).all() and (codes[bad][:, :70] == 0).all()
    assert np.array_equal(codes[[0, 3], :70], wc[[0, 3]]) and np.array_equal(scale[[0, 3]], wsc[[0, 3]])


@pytest.mark.gpu
@pytest.mark.parametrize("swiglu", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_rows_that_are_not_finite_among_many(dtype, swiglu):
    k, rows = 2320, 1300
    x = torch.randn(rows, k * (1 + swiglu), generator=torch.Generator().manual_seed(6)).to(DT[dtype])
    bad = np.array([0, 7, 500, 1299])
    for r, v in zip(bad, (float("nan"), float("inf"), float("-inf"), float("nan"))):
        x[r, (r * 37) % k] = v
    codes, scale, err = run_quantize(x.cuda(), k=k, swiglu=swiglu)
    good = np.setdiff1d(np.arange(rows), bad)
    assert err == 0 and np.isnan(scale[bad]).all() and not codes[bad].any() and np.isfinite(scale[good]).all()
    if not swiglu:
        wc, ws_ = plain_quantize(x[torch.from_numpy(good)].double().numpy())
        assert np.array_equal(codes[good][:, :k], wc) and np.array_equal(scale[good], ws_)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,copies,k", [(1, 8, 6144), (37, 3, 100), (300, 8, 2100), (5, 32, 16), (1100, 2, 2304), (3, 40, 1500), (1030, 3, 1040)])
def test_quantize_to_places(T, copies, k, dtype):
    rng = np.random.default_rng(T)
    rows = T * copies + 3
    place = rng.permutation(rows)[:T * copies].astype(np.int32)
    place[rng.random(T * copies) < 0.2] = -1
    x = torch.from_numpy(rng.standard_normal((T, k))).to(DT[dtype])
    wc, wsc = plain_quantize(x.double().numpy())

    def check(p, err):
        codes, scale, got = run_quantize(x.cuda(), place=torch.from_numpy(p).cuda(), copies=copies, rows=rows, ldc=up16(k) + 16)
        assert got == err
        want_c, want_s = np.full((rows, up16(k) + 16), -99, np.int8), np.full(rows, -7.0, np.float32)
        for s, to in enumerate(p):
            if 0 <= to < rows:
                want_c[to, :up16(k)] = 0
                want_c[to, :k], want_s[to] = wc[s // copies], wsc[s // copies]
        assert np.array_equal(codes, want_c) and np.array_equal(scale, want_s)
    check(place, 0)
    for worst in (rows, -2, -2 ** 31, 2 ** 31 - 1):
        p = place.copy()
        p[T * copies // 2] = worst
        check(p, q.DEVERR_GROUPING)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_strides(dtype):
    """Rows further apart, at addresses that are multiples of 32 and 16 bytes and of the element alone."""
    item = 4 if dtype == "f32" else 2
    for off, ld in ((0, 352), (16 // item, 352), (1, 352), (0, 349), (3, 351), (0, 344)):
        flat = torch.randn(off + 21 * ld, generator=torch.Generator().manual_seed(off + ld)).to(DT[dtype]).cuda()
        x = flat[off:].view(21, ld)
        for k in (336, 331):
            check_quantize(x[:, :k])
        check_swiglu(x, 160)
        check_swiglu(x, 171)


def check_swiglu(x, k):
    """float32 values a few units of their last place off: 8 of 2^-23 in the exponential's argument, quotient and
    product together, for gates within [-20, 20]; so codes lie within half a step of the value and that."""
    codes, scale, err = run_quantize(x, k=k, swiglu=1)
    v = x.double().cpu().numpy()
    gate, up = v[:, :k], v[:, k:2 * k]
    h = gate / (1 + np.exp(-gate)) * up
    off = 2.0 ** -20 * np.abs(h)
    m = np.maximum(np.abs(h).max(1), TINY)
    assert err == 0 and (np.abs(scale - m / 127) <= 2.0 ** -19 * m / 127).all()
    got = codes[:, :k] * scale[:, None].astype(np.float64)
    assert (np.abs(got - h) <= scale[:, None] / 2 * (1 + 2.0 ** -15) + off).all()
    assert (codes[:, k:up16(k)] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 2048), (7, 100), (130, 1024), (3, 4999), (2, 10000), (2, 6001), (1030, 1040), (1100, 2048), (1024, 1001)])
def test_quantize_swiglu(rows, k, dtype):
    g = torch.Generator().manual_seed(rows + k)
    check_swiglu((torch.randn(rows, 2 * k, generator=g) * 3).to(DT[dtype]).cuda(), k)


@pytest.mark.gpu
def test_quantize_swiglu_extremes():
    gate = torch.tensor([0.0, -0.0, 1e-40, 300.0, -300.0, 80.0, -80.0, 1.0])
    up = torch.tensor([5.0, 1.0, 1.0, 2.0, 7.0, -2.0, 1.0, -300.0])
    codes, scale, err = run_quantize(torch.cat([gate, up])[None].cuda(), k=8, swiglu=1)
    # gates far below 0 leave nothing, far above themselves: 600 is the largest
    want = np.rint(np.array([0, 0, 0, 600, 0, -160, 0, -300 / (1 + np.exp(-1))]) * 127 / 600)
    assert err == 0 and np.array_equal(codes[0, :8], want)
    for gv, uv in ((float("nan"), 1.0), (1.0, float("nan")), (float("inf"), 1.0), (1.0, float("-inf")), (0.0, float("inf")), (3e38, 3e38),
                   (float("-inf"), 1.0)):
        x = torch.cat([gate, up])[None].repeat(2, 1)
        x[1, 2], x[1, 10] = gv, uv
        codes, scale, _ = run_quantize(x.cuda(), k=8, swiglu=1)
        assert np.isnan(scale[1]) and not codes[1, :8].any() and np.array_equal(codes[0, :8], want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [48, 70, 1040, 2400, 13000])
def test_quantize_swiglu_far_gates(k, dtype):
    """Gates where 1 + exp(-gate) leaves float32 or the range of its fast quotients while SiLU(gate) * up does not: rows of such gates
    alone, whose products set the scale, and among others."""
    rng = np.random.default_rng(k)
    rows = []
    for lo in (-79.0, -80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -95.0, -104.0, -120.0, -150.0, -172.0, -177.0, -181.0, -300.0, -3e38):
        gate = lo + (rng.random(k) * 1.5 - 1.0 if lo > -1e3 else np.zeros(k))
        for size in (1e30, 3e38):
            rows.append(np.concatenate([gate, size * (0.05 + 0.95 * rng.random(k)) * rng.choice([-1, 1], k)]))
    for size in (1.0, 1e30):
        gate, up = rng.standard_normal(k) * 3, rng.standard_normal(k) * 3
        gate[::7], up[::7] = -80 - 15 * rng.random(len(gate[::7])), size * rng.random(len(up[::7])) * 1e6
        rows.append(np.concatenate([gate, up]))
    x = torch.from_numpy(np.stack(rows)).to(DT[dtype])
    check_swiglu(x.cuda(), k)
    if k < 3000:                                      # and where rows are many
        check_swiglu(x.repeat(40, 1).cuda(), k)
    # at -87.5 and -88.5 by itself, as the largest of the row
    y = torch.zeros(2, 2 * k)
    y[:, :k] = -1.0
    y[0, 5], y[0, k + 5] = -87.5, 1e30
    y[1, 5], y[1, k + 5] = -88.5, 1e30
    y = y.to(DT[dtype])
    codes, scale, err = run_quantize(y.cuda(), k=k, swiglu=1)
    g, u = y[:, 5].double().numpy(), y[:, k + 5].double().numpy()
    m = np.abs(g / (1 + np.exp(-g)) * u)
    assert err == 0 and (codes[:, 5] == -127).all() and (np.abs(scale - m / 127) <= 2.0 ** -19 * m / 127).all()


# ------------------------------------------------------------------ product


class Product:
    """Random codes for groups of the given rows, and the exact sums."""

    def __init__(self, counts, n, k, scales="random", tail=0, seed=0, pad=0, low=-128):
        rng = np.random.default_rng(seed + n * 7 + k)
        self.counts, self.n, self.k, self.rows = counts, n, k, sum(counts) + tail
        E, ld = len(counts), up16(k) + pad
        dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
        self.a = rng.integers(low, 128, (self.rows, k)).astype(np.int8)
        self.w = rng.integers(low, 128, (E, n, k)).astype(np.int8)
        ap, wp = rng.integers(-128, 128, (self.rows, ld)).astype(np.int8), rng.integers(-128, 128, (E, n, ld)).astype(np.int8)
        ap[:, :k], wp[:, :, :k] = self.a, self.w              # (what lies behind a row's values is not read)
        if scales == "random":
            self.sa, self.sw = (rng.random(self.rows) * 2e-2 + 1e-3).astype(np.float32), (rng.random((E, n)) * 2e-3 + 1e-4).astype(np.float32)
        elif scales == "powers":
            self.sa, self.sw = (np.ldexp(1.0, rng.integers(-9, 9, s)).astype(np.float32) for s in ((self.rows,), (E, n)))
        else:
            self.sa = self.sw = None
        self.off = np.concatenate([[0], np.cumsum(counts)])
        self.d_off = dev(self.off.astype(np.int32))
        self.d_a, self.d_w = dev(ap), dev(wp)
        self.d_sa, self.d_sw = (None, None) if self.sa is None else (dev(self.sa), dev(self.sw))

    def call(self, out, offsets=True, stream=None):
        W = ws()
        q.coli_moe_i8_product(q.i8_rows_for(self.d_a, self.d_sa), q.i8_mats_for(self.d_w, self.d_sw), self.k,
                              (self.d_off if offsets is True else offsets), 0 if out.dtype == torch.float32 else 1, out, out.stride(0), W, stream=stream)
        return W

    def want(self):
        v = np.zeros((self.off[-1], self.n))
        for e, (lo, hi) in enumerate(zip(self.off[:-1], self.off[1:])):
            s = self.a[lo:hi].astype(np.float64) @ self.w[e].astype(np.float64).T      # exact: below 2^53
            if self.sa is not None:
                s = s * self.sa[lo:hi, None].astype(np.float64) * self.sw[e].astype(np.float64)
            v[lo:hi] = s
        return v

    def check(self, dtype="f32", ldo=None, off=0, offsets=True):
        ldo = ldo or self.n
        flat = torch.full((off + self.rows * ldo + 8,), -7.0, dtype=DT[dtype], device="cuda")
        out = flat[off:off + self.rows * ldo].view(self.rows, ldo)[:, :self.n]
        W = self.call(out, offsets)
        assert q.coli_moe_error_word(W) == 0
        got, v = out.double().cpu().numpy(), self.want()
        tol = 3 * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0)
        assert (np.abs(got[:len(v)] - v) <= tol * 1.01 * np.abs(v)).all()
        out[:len(v)] = -7.0
        assert (flat == -7.0).all()                            # rows behind the groups, and what lies between rows
        return got[:len(v)], v


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts,n,k", [
    ([1], 1, 1), ([1], 128, 128), ([8], 256, 256), ([3], 130, 33), ([1], 4096, 6144), ([32], 100, 1000), ([33], 200, 129), ([70], 384, 500),
    ([1] * 8, 500, 300), ([0, 5, 0, 3, 1, 0], 131, 127), ([16, 17, 0, 15, 1, 31], 257, 320), ([40, 0, 90, 1, 129], 300, 161),
    ([200] + [0] * 19 + [3], 300, 200), ([300, 10, 200, 0, 257], 260, 145), ([1000], 700, 640), ([513], 1001, 31), ([2, 600], 513, 257)])
def test_product(counts, n, k, dtype):
    for scales in ("random", None):
        p = Product(counts, n, k, scales, tail=3)
        one = len(counts) == 1
        p.check(dtype)
        if one:
            p = Product(counts, n, k, scales)
            p.check(dtype, offsets=None)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[9], [20, 40, 0, 50], [300, 0, 280]])
def test_product_exact(counts):
    """Sums of at most 24 bits and scales that are powers of two: the very values."""
    for k in (96, 500, 1000):
        got, v = Product(counts, 140, k, "powers", tail=2).check()
        assert np.array_equal(got, v)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[5, 20], [60, 50, 0], [400, 130]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_product_strides(counts, dtype):
    for n, ldo, off, pad in ((136, 136, 0, 16), (136, 200, 8, 0), (135, 137, 1, 48), (136, 140, 0, 0), (250, 251, 0, 0)):
        Product(counts, n, 200, "random", tail=1, pad=pad).check(dtype, ldo, off)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 40, 200])
def test_product_longest_rows(rows):
    """The longest rows of the largest codes: sums up to 2^31 - 2^14."""
    k = 131071
    a = torch.full((rows, up16(k)), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, 8, up16(k)), -128, dtype=torch.int8, device="cuda")
    w[0, 1::2] = 127
    out, W = torch.empty(rows, 8, device="cuda"), ws()
    q.coli_moe_i8_product(q.i8_rows_for(a), q.i8_mats_for(w), k, None, 0, out, 8, W)
    want = np.tile(np.array([k * 16384, -k * 127 * 128], np.float32), 4)
    assert q.coli_moe_error_word(W) == 0 and (out.cpu().numpy() == want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[6], [50, 30], [300]])
def test_product_scales_out_of_the_usual_range(counts):
    """Scales whose product leaves float32's range while the result does not."""
    p = Product(counts, 72, 64, None, low=-127)
    rows = p.rows
    rng = np.random.default_rng(1)
    e = rng.integers(-126, 118, rows)
    f = rng.integers(-126, 118, (len(counts), 72))
    p.sa, p.sw = np.ldexp(1 + rng.random(rows), e).astype(np.float32), np.ldexp(1 + rng.random(f.shape), f).astype(np.float32)
    p.d_sa, p.d_sw = torch.from_numpy(p.sa).cuda(), torch.from_numpy(p.sw).cuda()
    out = torch.empty(rows, 72, device="cuda")
    W = p.call(out)
    got, v = out.double().cpu().numpy(), p.want()
    assert q.coli_moe_error_word(W) == 0
    big, small = np.abs(v) > 3.4028e38, np.abs(v) < 2.0 ** -125
    fine = ~big & ~small
    assert min(fine.sum(), big.sum(), small.sum()) > 20       # of 432 at least: all three kinds are there
    assert (np.abs(got - v)[fine] <= 3.1 * 2.0 ** -24 * np.abs(v)[fine]).all()
    assert (np.abs(got[big]) >= 3.4e38).all() and (np.sign(got[big]) == np.sign(v[big])).all()
    assert (np.abs(got - v)[small] <= 2.0 ** -147).all()
    # a row's scale of NaN is its row's alone, an infinite one too
    p.d_sa[0], p.d_sa[3] = float("nan"), 1.0
    p.call(out)
    assert torch.isnan(out[0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("scale,n,k", [(1, 72, 96), (12, 72, 96), (12, 72, 2700), (30, 1000, 2700)])
@pytest.mark.parametrize("bad", [[0, 5, 3, 28], [0, 5, 25, 1000], [-1, 5, 25, 28], [25, 5, 20, 28], [30, 31, 32, 33], [3, 3, 3, 2], [0, 37, 0, 37]])
def test_product_bad_offsets(scale, n, k, bad):
    """A group is left out where its own bounds are not ascending within the rows; every other one is multiplied, also
    where groups overlap and make more tiles than their rows would."""
    p = Product([5 * scale, 20 * scale, 3 * scale], n, k, None, tail=9 * scale)
    y = [p.a.astype(np.float64) @ w.astype(np.float64).T for w in p.w]
    off = [v * scale if v < 1000 else v * 1000 for v in bad]
    out = torch.full((p.rows, n), -7.25, device="cuda")
    W = p.call(out, torch.tensor(off, dtype=torch.int32, device="cuda"))
    good = [0 <= off[e] <= off[e + 1] <= p.rows for e in range(3)]
    assert q.coli_moe_error_word(W) == (0 if all(good) else q.DEVERR_GROUPING)
    got = out.cpu().numpy().astype(np.float64)
    for r in range(p.rows):
        claims = [e for e in range(3) if good[e] and off[e] <= r < off[e + 1]]
        if claims:
            assert np.any([got[r] == y[e][r] for e in claims], axis=0).all(), (r, claims)
        else:
            assert (got[r] == -7.25).all(), r


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 50, 150])
def test_product_far_apart(rows):
    """Matrices and result rows more than 2^32 bytes apart."""
    k, n = 64, 40
    gap = (1 << 32) + 4096
    store = torch.empty(2 * gap, dtype=torch.int8, device="cuda")
    w = store.as_strided((2, n, k), (gap, k, 1))
    p = Product([rows, rows], n, k, None)
    w.copy_(p.d_w)
    ld = ((1 << 32) + 64) // rows // 2 * 2
    out = torch.empty(2 * rows * ld, dtype=torch.bfloat16, device="cuda").view(2 * rows, ld)
    W = ws()
    q.coli_moe_i8_product(q.i8_rows_for(p.d_a), q.i8_mats_for(w), k, p.d_off, 1, out, ld, W)
    got, v = out[:, :n].double().cpu().numpy(), p.want()
    assert q.coli_moe_error_word(W) == 0 and (np.abs(got - v) <= 2.0 ** -8 * 1.01 * np.abs(v)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("counts,n,k", [([1], 12288, 2000), ([9], 12200, 2100), ([20], 12288, 2300), ([2, 1, 0, 5, 1, 1, 1, 3], 4096, 1500)])
def test_product_several_tiles_to_a_split(counts, n, k):
    """Few rows, more tiles than there are clusters that split k: every cluster takes several."""
    Product(counts, n, k, "random", tail=1).check()


@pytest.mark.gpu
def test_product_many_matrices():
    counts = [(i * 7) % 3 if i % 5 else 0 for i in range(1024)]
    Product(counts, 40, 48, "random", tail=2).check()


@pytest.mark.gpu
def test_two_streams_and_a_graph():
    """Products on two streams at once with a workspace each; a linear layer captured and replayed on new rows."""
    a, b = Product([300, 5, 100], 500, 700, "random"), Product([7, 8], 3000, 2000, "random", seed=1)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = torch.zeros(a.rows, 500, device="cuda"), torch.zeros(b.rows, 3000, device="cuda")
    torch.cuda.synchronize()
    words = []
    for _ in range(5):
        words += [a.call(o1, stream=s1), b.call(o2, stream=s2)]
    torch.cuda.synchronize()
    assert all(q.coli_moe_error_word(w) == 0 for w in words)
    for p, o in ((a, o1), (b, o2)):
        v = p.want()
        assert (np.abs(o.double().cpu().numpy() - v) <= 3.1 * 2.0 ** -24 * np.abs(v)).all()
    x, codes, scale = torch.zeros(20, 700, device="cuda"), torch.zeros(20, 704, dtype=torch.int8, device="cuda"), torch.zeros(20, device="cuda")
    out, W = torch.zeros(20, 500, device="cuda"), ws()
    rows, mats = q.i8_rows_for(codes, scale), q.i8_mats_for(a.d_w[:1], a.d_sw[:1])

    def linear():
        q.coli_moe_i8_quantize(0, 0, x, 20, 700, 700, None, 1, 20, codes, 704, scale, W)
        q.coli_moe_i8_product(rows, mats, 700, None, 0, out, 500, W)
    with torch.cuda.stream(s1):
        linear()
        s1.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s1):
            linear()
        for seed in range(3):
            x.copy_(torch.randn(20, 700, generator=torch.Generator().manual_seed(seed)))
            graph.replay()
            c, s = plain_quantize(x.double().cpu().numpy())
            v = (c.astype(np.float64) @ a.w[0].astype(np.float64).T) * s[:, None].astype(np.float64) * a.sw[0].astype(np.float64)
            assert (np.abs(out.double().cpu().numpy() - v) <= 3.1 * 2.0 ** -24 * np.abs(v)).all()
    assert q.coli_moe_error_word(W) == 0


# ------------------------------------------------------------------ together


@pytest.mark.gpu
@pytest.mark.parametrize("name,T", [("tiny", 8), ("olmoe", 1), ("olmoe", 300)])
def test_expert_half_over_int8_records(name, T):
    """Routing, sorted slots, both products straight from int8 records, SwiGLU, the weighted sum: every step against
    64-bit arithmetic on the step before it, the whole against the layer's own expert half."""
    wl = synth.WORKLOADS[name].replace(fmt=8, n_shared=0, shared_inter=0, act="bf16")
    H, I, E, K = wl.hidden, wl.inter, wl.n_experts, wl.top_k
    rec = synth.make_expert_records(wl, device="cuda")
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).cuda()
    router = q.MoERouter(E, K, wl.n_group, wl.topk_group, q.COLI_SCORE_SIGMOID, q.COLI_GROUP_TOP2, 1, 0, wl.routed_scaling)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    n = T * K
    ids, w = i32(n), torch.empty(T, K, device="cuda")
    q.coli_moe_route_scores(router, torch.randn(T, E, generator=torch.Generator().manual_seed(1)).cuda(), 0, None, T, ids, w)
    offsets, perm, place, W = i32(E + 1), i32(n), i32(n), ws()
    q.coli_moe_sort_rows(E, K, 1, None, T, H, 0, ids, offsets, perm, place, None, 0, W)

    lay = synth.record_layout(H, I, 8)
    stride = lay["stride"]
    w1 = rec.view(torch.int8).as_strided((E, 2 * I, H), (stride, H, 1), lay["wg"])
    wd = rec.view(torch.int8).as_strided((E, H, I), (stride, I, 1), lay["wd"])
    f = rec.view(torch.float32)
    s1, sd = f.as_strided((E, 2 * I), (stride // 4, 1), lay["sg"] // 4), f.as_strided((E, H), (stride // 4, 1), lay["sd"] // 4)
    xc, xs = torch.empty(n, H, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    q.coli_moe_i8_quantize(1, 0, x, T, H, H, place, K, n, xc, H, xs, W)
    gu = torch.empty(n, 2 * I, dtype=torch.bfloat16, device="cuda")
    q.coli_moe_i8_product(q.i8_rows_for(xc, xs), q.i8_mats_for(w1, s1), H, offsets, 1, gu, 2 * I, W)
    hc, hs = torch.empty(n, I, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    q.coli_moe_i8_quantize(1, 1, gu, n, 2 * I, I, None, 1, n, hc, I, hs, W)
    y = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")
    q.coli_moe_i8_product(q.i8_rows_for(hc, hs), q.i8_mats_for(wd, sd), I, offsets, 1, y, H, W)
    out = torch.empty(T, H, device="cuda")
    q.coli_moe_combine(1, y, n, H, place, w, T, K, H, 0, None, 0, out, H, W)
    assert q.coli_moe_error_word(W) == 0

    c, s = plain_quantize(x.double().cpu().numpy())
    slot = perm.cpu().numpy()
    assert np.array_equal(np.sort(slot), np.arange(n)) and np.array_equal(xc.cpu().numpy(), c[slot // K]) and np.array_equal(xs.cpu().numpy(), s[slot // K])
    off = offsets.tolist()
    for codes, scales, mats, mscale, got in ((xc, xs, w1, s1, gu), (hc, hs, wd, sd, y)):
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            if lo < hi:
                v = (codes[lo:hi].double() @ mats[e].double().t()) * scales[lo:hi, None].double() * mscale[e].double()
                assert ((got[lo:hi].double() - v).abs() <= (2.0 ** -8 + 2.0 ** -22) * v.abs()).all()
    h = torch.nn.functional.silu(gu[:, :I].double()) * gu[:, I:].double()
    assert ((hc.double() * hs.double()[:, None] - h).abs() <= hs.double()[:, None] * 0.50002 + 2.0 ** -20 * h.abs()).all()
    terms = y.double()[place.long()].view(T, K, H) * w.double()[:, :, None]
    assert ((out.double() - terms.sum(1)).abs() <= K * 2.0 ** -24 * terms.abs().sum(1)).all()

    # The layer's expert half rounds x and h to 16 bits or none.  8-bit steps are m / 127 with m about 4 deviations of x and
    # 10 of h: errors of 4 / 127 / sqrt(12) = 1% and 2.3% of a deviation, bf16's 0.2% twice; together below 3% of the
    # output's deviation, whose largest difference in a row is about 4 times that and whose largest value 3 to 4 deviations
    cfg = q.config_for(wl)
    counts, uniq, nu = i32(E), i32(E), i32(1)
    big = torch.empty(q.coli_moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    q.coli_moe_clear_error(big)
    q.coli_moe_group(cfg, ids, T, counts, i32(E + 1), i32(n), uniq, nu, big)
    ref = torch.empty(T, H, device="cuda")
    weights = q.weights_for(torch.zeros(E, H, device="cuda"), torch.zeros(E, device="cuda"), rec)
    q.coli_moe_ffn(cfg, weights, x, T, w, offsets, perm, uniq, nu, ref, big)
    assert q.coli_moe_error_word(big) == 0
    assert ((out - ref).abs().amax(1) <= 0.06 * ref.abs().amax(1)).all()
