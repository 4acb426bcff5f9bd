"""Sorted rows, combine, its gradient and 8-bit rows where the last row lies more than 2^32 bytes behind the first."""
import numpy as np
import pytest
import torch

from test_i8 import plain_quantize, up16
from test_sorted_rows import ACT, DT, Batch, check_grad, plain_sort, ws

q = pytest.importorskip("quantized_routed_expert_noaux_b200")


def far(n, h, dtype, unit):
    """n rows of h elements (not filled), `unit` elements the divisor of their distance, 2^32 bytes from the first to the last."""
    item = torch.empty(0, dtype=dtype).element_size()
    ld = ((1 << 32) // item // (n - 1) // unit + 1) * unit
    assert ld >= h and (n - 1) * ld * item > 1 << 32
    return torch.empty((n - 1) * ld + h, dtype=dtype, device="cuda").as_strided((n, h), (ld, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,hidden,unit", [(300, 64, 16), (300, 33, 1), (2700, 64, 16), (2700, 2064, 16), (2700, 33, 1), (2700, 2050, 2)])
def test_sort(T, hidden, unit, dtype):
    E, K = 16, 1
    ids = np.random.default_rng(T).integers(0, E, (T, K))
    x, rows = far(T, hidden, DT[dtype], unit), far(T, hidden, DT[dtype], unit)
    x.copy_(torch.randn(T, hidden, generator=torch.Generator().manual_seed(T)))
    rows.fill_(-7.0)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    offsets, perm, place, w = i32(E + 1), i32(T), i32(T), ws()
    q.coli_moe_sort_rows(E, K, ACT[dtype], x, T, hidden, x.stride(0), torch.from_numpy(ids).int().cuda(), offsets, perm, place, rows, rows.stride(0), w)
    wo, wp, wl, _ = plain_sort(ids, E)
    assert q.coli_moe_error_word(w) == 0 and np.array_equal(offsets.cpu().numpy(), wo) and np.array_equal(perm.cpu().numpy(), wp)
    assert np.array_equal(place.cpu().numpy(), wl) and torch.equal(rows.cpu(), x.cpu()[torch.from_numpy(wp)])


@pytest.mark.gpu
@pytest.mark.parametrize("act,out", [("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,hidden,unit", [(40, 64, 16), (40, 64, 4), (40, 33, 1), (2000, 264, 16), (2000, 333, 1)])
def test_combine_and_grad(T, hidden, unit, act, out):
    K = 2
    b = Batch(T, K, hidden, act, out)
    want = b.check()
    want_dy, want_dw = check_grad(b)
    y, o, add = far(b.rows, hidden, DT[act], unit), far(T, hidden, DT[out], unit), far(T, hidden, DT[out], unit)
    y.copy_(b.yv)
    add.copy_(b.add)
    W = ws()
    q.coli_moe_combine(ACT[act], y, b.rows, y.stride(0), b.d_place, b.d_w, T, K, hidden, ACT[out], add, add.stride(0), o, o.stride(0), W)
    assert np.array_equal(o.double().cpu().numpy(), want)
    add.copy_(b.dout)
    dy, dw = far(b.rows, hidden, DT[act], unit), torch.empty(T, K, device="cuda")
    dy.fill_(-7.0)
    q.coli_moe_combine_grad(ACT[act], y, b.rows, y.stride(0), b.d_place, b.d_w, T, K, hidden, ACT[out], add, add.stride(0), dy, dy.stride(0), dw, W)
    assert q.coli_moe_error_word(W) == 0 and torch.equal(dy, want_dy)
    # (rows of single elements may be summed by other threads than rows of 16-byte pieces)
    live = b.place >= 0
    terms = b.dout.double().numpy()[:, None] * b.y[np.maximum(b.place, 0)]
    assert torch.equal(dw, want_dw) or (np.abs(dw.double().cpu().numpy() - np.where(live, terms.sum(2), 0)) <= (hidden / 32 + 21) * 2.0 ** -24 * np.abs(terms).sum(2)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k,unit", [(50, 70, 16), (50, 3001, 1), (50, 48, 8), (1100, 2304, 16), (1100, 1001, 1)])
def test_quantize(rows, k, unit, dtype):
    x, codes = far(rows, k, DT[dtype], unit), far(rows, up16(k), torch.int8, 16)
    x.copy_(torch.randn(rows, k, generator=torch.Generator().manual_seed(k)))
    place = torch.from_numpy(np.random.default_rng(k).permutation(rows)).int().cuda()
    scale, w = torch.empty(rows, device="cuda"), ws()
    want_c, want_s = plain_quantize(x.double().cpu().numpy())
    for p in (None, place):
        codes.fill_(-99)
        q.coli_moe_i8_quantize(ACT[dtype], 0, x, rows, x.stride(0), k, p, 1, rows, codes, codes.stride(0), scale, w)
        at = np.arange(rows) if p is None else p.cpu().numpy()
        got = codes.cpu().numpy()[at]
        assert np.array_equal(got[:, :k], want_c) and not got[:, k:].any() and np.array_equal(scale.cpu().numpy()[at], want_s)
    assert q.coli_moe_error_word(w) == 0
