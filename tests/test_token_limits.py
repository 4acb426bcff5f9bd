"""How many tokens a layer takes at most."""
import pytest
import torch

q = pytest.importorskip("quantized_routed_expert_noaux_b200")


def refused(status, fn, *args, **kw):
    with pytest.raises(q.ColiError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status


@pytest.mark.parametrize("wfmt", [20, 36])
def test_tokens_beyond_the_gate_are_refused(wfmt):
    """The gate's tiles of 64 tokens are counted in 16 bits: 4,194,240 tokens are the most that the layer and
    the gate take, whatever else the shape allows."""
    cfg = q.MoEConfig(64, 64, 8, 1, 1, 1, 0, 64, 1.0, wfmt, 1, 0)
    n = q.coli_moe_record_bytes(64, 64, wfmt)
    w = q.MoEWeights(256, 256, 256, (n + 255) // 256 * 256, None)
    ws = torch.zeros(16, dtype=torch.uint8)  # too small: the check behind this one
    refused(7, q.coli_moe_layer, cfg, w, 256, 65535 * 64, 256, None, None, ws, stream=0)
    refused(4, q.coli_moe_layer, cfg, w, 256, 65535 * 64 + 1, 256, None, None, ws, stream=0)
    refused(4, q.coli_moe_gate, cfg, 256, 256, 65535 * 64 + 1, 256, stream=0)
    # the expert half has no gate
    refused(7, q.coli_moe_ffn, cfg, w, 256, 65535 * 64 + 1, 256, 256, 256, 256, 256, 256, ws, stream=0)
