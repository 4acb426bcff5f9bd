"""What the binding of the 4-bit operators refuses of tensors."""
import numpy as np
import pytest
import torch

from test_fp4 import Product
from test_fp4 import ws as workspace

q = pytest.importorskip("quantized_routed_expert_noaux_b200")


def refused(status, fn, *args, **kw):
    with pytest.raises(q.ColiError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status


@pytest.mark.parametrize("explicit", [False, True])
def test_any_tensor_off_the_gpu_is_refused(explicit):
    """Host tensors in any place of a call, with a stream given or not (device pointers as integers elsewhere)."""
    if torch.cuda.is_available():
        pytest.skip("host check: where it runs nothing could be launched on such a pointer")
    kw = {"stream": 0} if explicit else {}
    t = torch.zeros(64)

    def each(fn, args, places):
        for i in places:
            a = list(args)
            a[i] = t
            refused(1, fn, *a, **kw)
    r = q.MoERouter(8, 2, 1, 1, 0, 0, 1, 0, 1.0)
    each(q.coli_moe_route_scores, [r, 256, 0, 256, 1, 512, 1024], (1, 3, 5, 6))
    each(q.coli_moe_fp4_quantize, [0, 0, 0, 256, 1, 32, 256, 1, 1, 32, 256, 256, 256, 256], (3, 6, 10, 11, 12, 13))
    each(q.coli_moe_fp4_dequantize, [0, 0, 256, 256, 256, 1, 32, 0, 256, 32], (2, 3, 4, 8))
    a, w = q.FP4Rows(256, 256, 256, 1), q.FP4Mats(256, 256, 256, 1, 8, 0, 0, 0)
    each(q.coli_moe_fp4_product, [0, a, w, 32, 256, 0, 256, 8, 256], (4, 6, 8))
    each(q.coli_moe_fp4_pack_record, [q.MoEConfig(64, 64, 2, 1, 1, 1, 0, 64, 1.0, 20, 1, 0), 0, 256, 256, 256, 256, 256], (2, 3, 4, 5, 6))


def test_helpers_refuse_tensors_that_are_not_dense():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    codes, scales, row = u8(4, 64), u8(4, 16), torch.zeros(4)
    refused(2, q.fp4_rows_for, u8(4, 128)[:, :64], scales, row)
    refused(2, q.fp4_rows_for, u8(64, 4).t(), scales, row)
    refused(2, q.fp4_rows_for, u8(8, 64)[::2], scales, row)
    refused(2, q.fp4_rows_for, codes, u8(4, 32)[:, ::2], row)
    refused(2, q.fp4_rows_for, codes, scales, torch.zeros(8)[::2])
    mats = u8(3, 8, 64), u8(3, 2048), torch.zeros(3, 8)
    refused(2, q.fp4_mats_for, u8(3, 8, 128)[:, :, :64], *mats[1:])
    refused(2, q.fp4_mats_for, u8(3, 16, 64)[:, ::2], *mats[1:])
    refused(2, q.fp4_mats_for, u8(3, 64, 8).transpose(1, 2), *mats[1:])
    refused(2, q.fp4_mats_for, mats[0], u8(3, 4096)[:, ::2], mats[2])
    refused(2, q.fp4_mats_for, mats[0], u8(3, 4, 1024)[:, :2], torch.zeros(3, 16)[:, ::2])
    refused(2, q.fp4_mats_for, mats[0], mats[1], torch.zeros(3, 16)[:, ::2])
    # dense, but not on a GPU
    refused(1, q.fp4_rows_for, codes, scales, row)
    refused(1, q.fp4_mats_for, *mats)


@pytest.mark.gpu
def test_helpers_take_matrices_further_apart():
    """The matrices of a stack may lie apart: records that hold their codes, scales and row scales one after another."""
    p = Product(1, [4, 0, 9], 72, 96, exact=True)
    c = p.dev[3:]
    apart = [torch.zeros(t.shape[0], 3 * t[0].numel() + (-3 * t[0].numel()) % 16, dtype=t.dtype, device="cuda") for t in c]
    views = [a[:, :t[0].numel()].unflatten(1, t.shape[1:]) for a, t in zip(apart, c)]
    for v, t in zip(views, c):
        v.copy_(t)
    out = torch.full((13, 72), -7.0, device="cuda")
    W = workspace()
    q.coli_moe_fp4_product(1, q.fp4_rows_for(*p.dev[:3]), q.fp4_mats_for(*views), 96, p.dev_offsets, 0, out, 72, W)
    assert q.coli_moe_error_word(W) == 0 and np.array_equal(out.double().cpu().numpy(), p.want()[0])


def test_operands_of_another_device_are_refused():
    """Structures of the helpers know their device: a product with operands of two, or of another than its result's."""
    if torch.cuda.is_available():
        pytest.skip("host check: where it runs nothing could be launched on such a pointer")
    a, w = q.FP4Rows(256, 256, 256, 1), q.FP4Mats(256, 256, 256, 1, 8, 0, 0, 0)
    a.device, w.device = 0, 1
    refused(1, q.coli_moe_fp4_product, 0, a, w, 32, None, 0, 256, 8, 256, stream=0)
