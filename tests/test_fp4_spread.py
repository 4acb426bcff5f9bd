"""Quantisation of rows that an index takes several times, around the sizes where every source row is quantised once
and copied, or every row by itself: the results are those of the source rows."""
import pytest
import torch

from test_fp4 import DT, run_quantize, test_quantize_many_copies as many_copies

q = pytest.importorskip("quantized_routed_expert_noaux_b200")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,div,k", [(400, 16, 2048), (333, 32, 1984), (150, 9, 1792), (90, 40, 4064), (200, 8, 2304), (700, 3, 512)])
def test_copies(fmt, dtype, T, div, k):
    """Permuted, taken mostly from one row, and with bad indices among them, against 64-bit arithmetic."""
    many_copies(fmt, dtype, T, div, k)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,div,k", [(30000, 2, 6144), (40000, 2, 6144), (20000, 8, 2048), (50000, 8, 1024), (9000, 4, 16384)])
def test_large_batches(fmt, dtype, T, div, k):
    """Against the source rows quantised one by one and gathered."""
    x = torch.randn(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(k + T)).to(DT[dtype])
    index = torch.randperm(T * div, device="cuda", generator=torch.Generator("cuda").manual_seed(T)).to(torch.int32)
    codes, scales, row, w = run_quantize(x, fmt, 0, index, div, T * div)
    c0, s0, r0, _ = run_quantize(x, fmt)
    src = (index // div).long()
    assert torch.equal(codes, c0[src]) and torch.equal(row, r0[src])
    assert torch.equal(scales.view(T * div, -1), s0.view(T, -1)[src])
    assert q.coli_moe_error_word(w) == 0
