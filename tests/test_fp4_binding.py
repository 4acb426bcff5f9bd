"""What the binding of the 4-bit operators refuses of tensors."""
import pytest
import torch

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
