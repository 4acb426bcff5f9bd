"""Which rows a grouped product writes under offsets that are not ascending."""
import numpy as np
import pytest
import torch

import _fp4 as ref
from test_fp4 import Product

q = pytest.importorskip("quantized_routed_expert_noaux_b200")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("scale", [1, 12])  # the rows of every group: single CTAs, and pairs of them
@pytest.mark.parametrize("bad", [[0, 5, 3, 28], [0, 5, 25, 1000], [-1, 5, 25, 28], [25, 5, 20, 28], [30, 31, 32, 33], [3, 3, 3, 2]])
def test_rows_written_under_bad_offsets(fmt, scale, bad):
    """A group is left out where its own bounds are not ascending within the rows; every other group is
    multiplied as it stands.  Rows that two groups claim hold one's product or the other's."""
    p = Product(fmt, [5 * scale, 20 * scale, 3 * scale], 72, 96, exact=True, tail=9 * scale)
    x = ref.values(*p.a, fmt)
    y = [x @ ref.values(*w, fmt).T for w in p.w]
    off = [v * scale if v < 1000 else v * 1000 for v in bad]
    out = torch.full((p.rows, 72), -7.0, device="cuda")
    w = p.call(out, 0, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    good = [0 <= off[e] <= off[e + 1] <= p.rows for e in range(3)]
    assert q.coli_moe_error_word(w) == (0 if all(good) else q.DEVERR_GROUPING)
    got = out.cpu().numpy().astype(np.float64)
    for r in range(p.rows):
        claims = [e for e in range(3) if good[e] and off[e] <= r < off[e + 1]]
        if claims:
            assert np.any([got[r] == y[e][r] for e in claims], axis=0).all(), (r, claims)
        else:
            assert (got[r] == -7.0).all(), r
