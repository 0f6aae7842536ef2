"""The training operators on the GPU where one value of a row, a block or a call is unlike the others: a NaN among masked
choices, biases whose sums pass fp32, gradients whose squares are almost nothing or too much, memory that a tensor lets go.
Definitions and tolerances are those of test_gpu_train."""

import math

import pytest
import torch

from tests import test_gpu_train as H
from tests.test_gpu_train import BF16, F16, F32, km  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


# ---- routing ----------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("negative", [False, True])
@pytest.mark.parametrize("K", [8, 100, 2048, 2050, 4096])
def test_route_of_a_nan_among_masked_choices(km, K, negative, dt):  # noqa: F811
    """The row has no scores, wherever the NaN is and whatever its sign: also among choices of which only masked ones share
    its lane."""
    n = 24
    x = torch.full((n, K), -math.inf, dtype=dt)
    g = H.gen(K)
    for row in range(n):
        at = torch.randperm(K, generator=g)[:4]
        x[row, at[:3]] = torch.randn(3, generator=g).to(dt)
        x[row, at[3]] = math.nan
        if row % 4 == 3:  # rows without one, and with the NaN alone
            x[row, at[3]] = 0.5
        elif row % 8 == 6:
            x[row, at[:3]] = -math.inf
    if negative:
        kind = torch.int32 if dt == F32 else torch.int16
        bits = x.view(kind)
        bits[torch.isnan(x)] |= torch.iinfo(kind).min
    assert bool(torch.isnan(x).any(-1)[0]) and bool((torch.signbit(x[torch.isnan(x)]) == negative).all())
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            for S in (1, 2, 5):
                got = km.route(x.cuda(), S, score=score, renormalise=renormalise)
                H.check_route(got, x, S, score=score, renormalise=renormalise)


# ---- AdamW ------------------------------------------------------------------------------------------------------------
