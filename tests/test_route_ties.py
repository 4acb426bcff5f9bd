"""Routing from float32 and bf16 logits that are equal, or differ by less than float32's smallest normal
number, where a lane holds several experts: the order is that of the logits, ties go to the lower id."""
import pytest
import torch

from test_route_scores import INF, MAXG, SIG, SOFT, TOP2, check, router


def rows_of(E, dtype):
    """Rows of logits near zero: the tied or nearly tied experts lie in different lanes at different places."""
    g = torch.Generator().manual_seed(E)
    per = (E + 31) // 32
    r = torch.full((14, E), -1.0)
    r[0, 3], r[0, per] = 0.0, 0.0                                # two zeros: place 3 of lane 0, place 0 of lane 1
    r[1, [1, per + 2 if per > 2 else per, E - 1]] = 0.0
    r[2] = 0.0
    r[3] = -0.0
    r[3, ::3] = 0.0                                              # zeros of both signs are one value
    r[4] = torch.where(torch.rand(E, generator=g) < 0.2, 0.0, -torch.rand(E, generator=g))     # ReLU-like, negated
    r[5] = -torch.relu(torch.randn(E, generator=g))              # shifted so that the largest is 0
    r[6] = 0.0
    r[6, E // 2:] = -INF
    tiny = torch.finfo(torch.float32).smallest_normal
    step = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133                   # one unit of a subnormal
    order = torch.randperm(E, generator=g).double()
    r[7] = (order * step).float()                                # subnormals one unit apart, in any order
    r[8] = -r[7]
    r[9] = (torch.arange(E).double() * step).float()             # ascending ids
    r[10] = ((torch.arange(E).double() - E // 2) * step).float()  # across zero
    r[11] = ((order % 5) * step).float()                         # subnormals with ties
    r[12] = (tiny + ((order % 7) - 3) * step).float()            # around the smallest normal number
    r[13] = torch.where(torch.rand(E, generator=g) < 0.5, 0.0, step * 1.0).float()
    return r.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,TG", [(40, 1, 1), (64, 1, 1), (64, 4, 2), (160, 8, 3), (256, 1, 1), (256, 8, 4), (1000, 1, 1), (1024, 1, 1), (1024, 32, 5)])
def test_ties_near_zero(score, dtype, E, G, TG):
    rows = rows_of(E, dtype)
    act = 0 if dtype == torch.float32 else 1
    for K in (1, 2, 7, 8):
        for group in (MAXG, TOP2):
            check(rows, None, router(E, K, G, TG, score, group, 1, act))
    check(rows, None, router(E, 5, G, TG, score, MAXG, 0, act))


@pytest.mark.gpu
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("E,G,TG", [(64, 4, 2), (256, 8, 4), (1024, 1, 1)])
def test_ties_of_ordinary_values(score, E, G, TG):
    """The same where the tied values are ordinary, of both signs and across a power of two, with and without a
    bias of zeros."""
    g = torch.Generator().manual_seed(E + 1)
    rows = torch.randint(-2, 3, (6, E), generator=g).float()
    rows[1] += 1.0
    rows[2] = torch.where(torch.rand(E, generator=g) < 0.5, 1.0, 1.0 - 2.0 ** -24)
    rows[3] = -rows[2]
    rows[4] = 2.0 ** 20 + torch.randint(0, 3, (E,), generator=g) * 2.0 ** -3
    for K in (1, 2, 8):
        for bias in (None, torch.zeros(E)):
            check(rows, bias, router(E, K, G, TG, score, MAXG, 1))
