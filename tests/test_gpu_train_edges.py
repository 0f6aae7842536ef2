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


def test_route_of_group_sums_past_fp32(km):  # noqa: F811
    """Two groups whose worths both overflow 32 bits are told apart in 64; a worth of +inf is larger than either."""
    K, G = 32, 8
    x = H.some_logits(40, K, F32, 3)
    for values in ([2e38, 2e38, 3e38, 3e38], [3e38, 1e38, 2e38, 3e38], [2e38, 2e38, math.inf, 0.0], [math.inf, -1e38, math.inf, 3e38],
                   [-3e38, -3e38, -2e38, -2e38]):
        for first in (0, 12):
            bias = torch.zeros(K) if values[0] > 0 else torch.full((K,), -3.2e38)
            bias[first:first + 2] = torch.tensor(values[:2])
            bias[first + 8:first + 10] = torch.tensor(values[2:])
            for keep in (1, 2):
                for score in ("softmax", "sigmoid"):
                    kw = dict(score=score, groups=G, top_groups=keep, renormalise=False)
                    H.check_route(km.route(x.cuda(), 3, bias=bias.cuda(), **kw), x, 3, bias=bias, **kw)


# ---- AdamW ------------------------------------------------------------------------------------------------------------
