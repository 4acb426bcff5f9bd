"""Products of microscaled 4-bit operands whose row scales lie so far apart, or are so large or small, that their
product leaves float32's range while the result does not."""
import numpy as np
import pytest
import torch

import _fp4 as ref
from _rounding import to_bf16, to_f32
from test_fp4 import ws

q = pytest.importorskip("quantized_routed_expert_noaux_b200")


def operand(rng, rows, k, fmt, row):
    """Codes of every value under one block scale: sums of 1056 terms are exact in float32."""
    code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    byte = np.full((rows, k // ref.BLOCK[fmt]), 130 if fmt == 0 else 0x78, np.uint8)  # 8, or 256
    return code, byte, row.astype(np.float32)


def product(fmt, a, w, sizes, n, k, act):
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    rows = len(a[0])
    out = torch.full((rows, n), -7.0, dtype=torch.float32 if act == 0 else torch.bfloat16, device="cuda")
    keep = [dev(ref.pack(a[0])), dev(ref.rows_layout(a[1], fmt, k)), dev(a[2]), dev(np.stack([ref.pack(x[0]) for x in w])),
            dev(np.stack([ref.tiles_layout(x[1], fmt, k) for x in w])), dev(np.stack([x[2] for x in w]))]
    off = dev(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32))
    W = ws()
    q.coli_moe_fp4_product(fmt, q.fp4_rows_for(*keep[:3]), q.fp4_mats_for(*keep[3:]), k, off, act, out, n, W)
    assert q.coli_moe_error_word(W) == 0
    return out.double().cpu().numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 20], [40, 33], [150], [300, 130]])
@pytest.mark.parametrize("act", [0, 1])
def test_row_scales_far_apart(fmt, sizes, act):
    """Row scales from 2^-126 to 2^117 on both sides, in any order, beside ordinary ones; rows of zeros among
    them.  Sums are exact and scales powers of two, so results are the real ones rounded once, but that one
    below 2^-126 may be rounded twice (in float32 and to a type with as small an exponent)."""
    n, k = 136, 1056
    rows = sum(sizes)
    rng = np.random.default_rng(rows + fmt)
    a = operand(rng, rows, k, fmt, np.ldexp(1.0, rng.choice([-126, -110, -100, -20, 0, 30, 64, 100, 117], rows)))
    a[0][::5] &= 8                                        # rows of zeros of both signs
    w = [operand(rng, n, k, fmt, np.ldexp(1.0, rng.choice([-126, -90, -50, -12, 0, 25, 63, 64, 117], n))) for _ in sizes]
    got = product(fmt, a, w, sizes, n, k, act)
    lo = 0
    for size, m in zip(sizes, w):
        s = ref.values(*a[:2], None, fmt)[lo:lo + size] @ ref.values(*m[:2], None, fmt).T
        assert np.abs(s).max(initial=0) < 2.0 ** 36
        y = s * a[2][lo:lo + size, None].astype(np.float64) * m[2][None, :].astype(np.float64)
        want = to_f32(y) if act == 0 else to_bf16(y)
        g = got[lo:lo + size]
        small = np.abs(y) < 2.0 ** -126
        assert np.array_equal(g[~small], want[~small])
        # one unit of the type's subnormals
        assert (np.abs(g - y)[small] <= (2.0 ** -149 if act == 0 else 2.0 ** -133)).all()
        lo += size


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("sizes", [[7], [60], [260]])
def test_row_scales_of_any_significand(fmt, sizes):
    """The same with row scales that are no powers of two, subnormal ones and zeros: two roundings to float32,
    and one unit of its subnormals for each."""
    n, k = 136, 288
    rows = sizes[0]
    rng = np.random.default_rng(rows + 7 * fmt)
    def scales(count):
        s = (rng.random(count) + 1) * np.ldexp(1.0, rng.choice([-140, -126, -100, -64, -3, 0, 2, 64, 100, 126], count))
        s[rng.random(count) < 0.05] = 0.0
        return np.where(rng.random(count) < 0.3, -s, s)
    a, w = operand(rng, rows, k, fmt, scales(rows)), operand(rng, n, k, fmt, scales(n))
    got = product(fmt, a, [w], sizes, n, k, 0)
    s = ref.values(*a[:2], None, fmt) @ ref.values(*w[:2], None, fmt).T
    y = s * a[2][:, None].astype(np.float64) * w[2][None, :].astype(np.float64)
    over = np.abs(y) > 2.0 ** 128 * (1 - 2.0 ** -22)     # rounds to infinity, or may
    assert (np.abs(got[over]) >= np.finfo(np.float32).max * (1 - 2.0 ** -21)).all() and (np.sign(got[over]) == np.sign(y[over])).all()
    # a subnormal first rounding is followed by a factor below 2: three units of 2^-149 in all
    assert (np.abs(got - y)[~over] <= 2 * 2.0 ** -24 * 1.01 * np.abs(y)[~over] + 3 * 2.0 ** -149).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 50, 900])
def test_swiglu_of_zero_sums(T):
    """The expert half where gate and up sums are zero under row scales whose product leaves float32: x is
    2^110 in column 0 alone, the gate and up matrices are 2^100 everywhere but there; other tokens are
    ordinary.  The first tokens' h and result are zero, not NaN."""
    H, I, E = 256, 128, 2
    cfg = q.MoEConfig(H, I, E, 1, 1, 1, 0, I, 1.0, 20, 1, 0)
    n = q.coli_moe_record_bytes(H, I, 20)
    rec = torch.zeros(E, (n + 255) // 256 * 256, dtype=torch.uint8, device="cuda")
    W = ws()
    big = torch.full((I, H), 2.0 ** 100)
    big[:, :16] = 0.0
    g = torch.Generator().manual_seed(T)
    wd = torch.randn(H, I, generator=g)
    for e in range(E):
        q.coli_moe_fp4_pack_record(cfg, 0, big.cuda(), big.cuda(), wd.cuda(), rec[e], W)
    x = torch.zeros(T, H)
    x[::2, 0] = 2.0 ** 110
    x = x.to(torch.bfloat16).cuda()
    w = q.weights_for(None, None, rec)
    buf = torch.zeros(q.coli_moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    ids = (torch.arange(T) % E).to(torch.int32).reshape(T, 1).cuda()
    i32 = lambda m: torch.empty(m, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, offsets, perm, uniq, nu = i32(E), i32(E + 1), i32(T), i32(E), i32(1)
    q.coli_moe_group(cfg, ids, T, counts, offsets, perm, uniq, nu, buf)
    out = torch.full((T, H), -7.0, device="cuda")
    q.coli_moe_ffn(cfg, w, x, T, torch.ones(T, 1, device="cuda"), offsets, perm, uniq, nu, out, buf)
    assert q.coli_moe_error_word(buf) == 0
    assert (out == 0).all()
