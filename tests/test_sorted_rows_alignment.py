"""Combine and its gradient where rows start at odd multiples of 16 bytes: 8 bf16 values are 16 bytes of a row, but
32 of a float32 addend, result or gradient, and a load of 32 bytes wants a multiple of 32.

The sums are the same ones in the same order wherever the rows lie, so results are compared bit for bit with those of rows at
multiples of 32 bytes, and these with 64-bit arithmetic (test_sorted_rows)."""
import pytest
import torch

from test_sorted_rows import ACT, Batch, check_grad, rows_at, ws

q = pytest.importorskip("quantized_routed_expert_noaux_b200")

ITEM = {"f32": 4, "bf16": 2}
SHAPES = [(1, 8, 8), (3, 2, 6144), (37, 5, 64), (6000, 2, 72), (300, 10, 2056), (2048, 8, 1024)]
# of the addend, the result and dout: bytes from their storage's start to the first row, and beyond a row to the next one
WHERE = [(16, 0), (0, 16), (16, 16), (48, 48), (16, 32), (32, 16)]


def view_of(values, dtype, first, gap):
    """`values` on the GPU, row 0 `first` bytes into its storage, rows `gap` bytes further apart than their length."""
    item = ITEM[dtype]
    view = rows_at(values, values.shape[1] + gap // item, first // item, dtype)[1]
    assert view.data_ptr() % 32 == first % 32 and (view.shape[0] == 1 or view.stride(0) * item % 32 == (values.shape[1] * item + gap) % 32)
    return view


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,hidden", SHAPES)
def test_combine(T, K, hidden, act, out):
    b = Batch(T, K, hidden, act, out)
    b.check()
    aligned = torch.empty(T, hidden, dtype=rows_at(b.add[:1], hidden, 0, out)[1].dtype, device="cuda")

    def call(y, add, o):
        W = ws()
        q.coli_moe_combine(ACT[act], y, b.rows, y.stride(0), b.d_place, b.d_w, T, K, hidden, ACT[out], add, 0 if add is None else add.stride(0), o,
                           o.stride(0), W)
        assert q.coli_moe_error_word(W) == 0
        return o
    want = call(b.yv, b.add.cuda(), aligned).clone()
    bare = call(b.yv, None, aligned).clone()
    for where in WHERE:
        add = view_of(b.add, out, *where)
        o = view_of(torch.zeros(T, hidden), out, *where)
        assert torch.equal(call(b.yv, add, aligned), want)               # the addend alone lies there
        assert torch.equal(call(b.yv, b.add.cuda(), o), want)            # the result alone
        assert torch.equal(call(b.yv, add, o), want)
        assert torch.equal(call(b.yv, None, o), bare)
        assert torch.equal(call(b.yv, add, add), want)                   # in place
        y = view_of(b.yv.cpu(), act, *where)
        assert torch.equal(call(y, view_of(b.add, out, *where), o), want)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,hidden", SHAPES)
def test_grad(T, K, hidden, act, out):
    b = Batch(T, K, hidden, act, out)
    want_dy, want_dw = check_grad(b)
    for where in WHERE:
        dout = view_of(b.dout, out, *where)
        for y, dy in ((b.yv, torch.full_like(b.yv, -7.0)), (view_of(b.yv.cpu(), act, *where), view_of(torch.full((b.rows, hidden), -7.0), act, *where))):
            for has_dy, has_dw in ((True, True), (True, False), (False, True)):
                dw, W = torch.full((T, K), -7.0, device="cuda"), ws()
                dy.fill_(-7.0)
                q.coli_moe_combine_grad(ACT[act], y, b.rows, y.stride(0), b.d_place, b.d_w, T, K, hidden, ACT[out], dout, dout.stride(0),
                                        dy if has_dy else None, dy.stride(0) if has_dy else 0, dw if has_dw else None, W)
                assert q.coli_moe_error_word(W) == 0
                assert not has_dy or torch.equal(dy, want_dy)
                assert not has_dw or torch.equal(dw, want_dw)
