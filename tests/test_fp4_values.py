"""Values read back from microscaled 4-bit rows, over the whole range of block and row scales: the real value
rounded once to float32, and that to bf16."""
import numpy as np
import pytest
import torch

import _fp4 as ref
from _rounding import to_bf16, to_f32
from test_fp4 import ACT, DT

q = pytest.importorskip("quantized_routed_expert_noaux_b200")


def read_back(fmt, code, byte, row, dtype, layout=0):
    rows, k = code.shape
    lay = ref.rows_layout(byte, fmt, k).reshape(-1) if layout == 0 else ref.tiles_layout(byte, fmt, k)
    out = torch.full((rows, k), -7.0, dtype=DT[dtype], device="cuda")
    q.coli_moe_fp4_dequantize(fmt, layout, torch.from_numpy(ref.pack(code)).cuda(), torch.from_numpy(lay).cuda(),
                              torch.from_numpy(row.astype(np.float32)).cuda(), rows, k, ACT[dtype], out, k)
    return out.double().cpu().numpy()


def check_read_back(fmt, code, byte, row, layout=0):
    v = ref.values(code, byte, None, fmt) * row.astype(np.float32).astype(np.float64)[:, None]
    for dtype, rounded in (("f32", to_f32), ("bf16", lambda x: to_bf16(to_f32(x)))):
        got, want = read_back(fmt, code, byte, row, dtype, layout), rounded(v)
        assert np.array_equal(got, want, equal_nan=True), dtype


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("layout", [0, 1])
def test_row_scales_of_any_significand(fmt, layout):
    """Among them row scales under which the float32 value lies on the middle of two bf16 values while the real one
    does not."""
    rng = np.random.default_rng(3)
    rs = (rng.random(400000) + 1).astype(np.float32).astype(np.float64)
    picked = []
    for p in (3.0, 1.5, 6.0) if fmt == 0 else (3.0 * 1.125, 1.5 * 1.375, 3.0 * 1.625, 6.0 * 1.875):
        v = p * rs
        picked.append(rs[to_bf16(to_f32(v)) != to_bf16(v)])
    row = np.concatenate(picked + [rs[:40]])
    assert len(row) > 45                                    # some of them are such scales
    row = np.concatenate([row, -row, row * 2.0 ** -100])
    k = 512
    code = np.tile(np.arange(16, dtype=np.uint8), k // 16)[None, :].repeat(len(row), 0)
    byte = np.full((len(row), k // ref.BLOCK[fmt]), 127, np.uint8)
    if fmt == 1:
        byte[:] = 0x38 + np.arange(k // 16) % 8             # 1 .. 1.875
    check_read_back(fmt, code, byte, row, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("k", [64, 2080])
def test_values_at_the_ends_of_the_range(fmt, k):
    """Every code under every block scale, under row scales that bring values out of float32's range back
    into it, or near its subnormals."""
    row = np.array([1.0, 0.25, 2.0 ** -100, 2.0 ** -126, 1.3 * 2.0 ** -126, 1.7 * 2.0 ** -60, 2.0 ** 100, 1.1 * 2.0 ** 117, 2.0 ** 127, 1.9 * 2.0 ** 126, -3.1,
                    0.0, 2.0 ** -149, 5 * 2.0 ** -147, 2.0 ** -119, 1.0 + 2.0 ** -16, 1.0 + 2.0 ** -17, 2.0 ** -123 * (1 + 2.0 ** -16)])
    nb = 255 if fmt == 0 else 127
    bytes_ = np.arange(nb, dtype=np.uint8)
    block = ref.BLOCK[fmt]
    per = k // block
    groups = -(-nb // per)
    byte = np.resize(bytes_, groups * per).reshape(groups, per)
    code = np.tile(np.arange(16, dtype=np.uint8), k // 16)[None, :].repeat(groups, 0)
    check_read_back(fmt, np.tile(code, (len(row), 1)), np.tile(byte, (len(row), 1)), row.repeat(groups))
