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

@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_a_square_past_fp32(km, bits):  # noqa: F811
    """A gradient whose square is infinite stops its element, whatever else its block holds, and no other."""
    for others in (0.0, 1e-3):
        p = torch.ones(600, device="cuda")
        g = torch.full((600,), others, device="cuda")
        g[300] = 1e25
        M, V, scales = km.adamw_states([p], bits)
        plan = km.adamw_plan([p], [g], M, V, scales=scales)
        for step in (1, 2, 3):
            km.adamw(plan, lr=1e-2, step=step, weight_decay=0.0)
            g[300] = 0.0
            v = V[0].float() if bits == 8 else V[0]
            assert bool(torch.isfinite(p).all()) and float(p[300]) == 1.0, step
            assert float(v[300]) == math.inf and int(torch.isfinite(v).sum()) == 599
            if bits == 8:
                assert float(scales[1][0][1]) > 0
        # (beside an m of 1e24 the others' m is 0 in 8 bits: they have moved once)
        assert bool((p[:256] == p[0]).all()) and bool((p[512:] == p[0]).all()) and bool((p[0] < 1.0) == (others > 0))
        assert bool(((p[256:512] < 1.0) == (others > 0))[torch.arange(256) != 44].all())


@pytest.mark.parametrize("size", [1e-13, 3e-15, 1e-16, 1e-18])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-8])
def test_adamw_8bit_of_small_gradients(km, size, eps):  # noqa: F811
    """Gradients whose squares are next to nothing, then none: an element that has moved never divides by eps alone.  A step
    is off by half a step of m's code (2^-4) and half of that of v's (2^-3), and in 64 bits' terms by the rounding of v
    below the normal range (1e-39 in steps of 2^-149 = 1.4e-45: nothing beside them)."""
    n = 700
    u = 1.0 + 2.0 * torch.rand(n, generator=H.gen(1))
    g0 = (size * u).to(F32)
    p, g = torch.zeros(n, device="cuda"), g0.cuda()
    M, V, scales = km.adamw_states([p], 8)
    plan = km.adamw_plan([p], [g], M, V, scales=scales)
    m, v = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    b1, b2, lr = 0.9, 0.999, 0.25
    for step in range(1, 5):
        before = p.cpu().double()
        km.adamw(plan, lr=lr, step=step, betas=(b1, b2), eps=eps, weight_decay=0.0)
        gr = g0.double() if step == 1 else 0.0
        m, v = b1 * m + (1 - b1) * gr, b2 * v + (1 - b2) * gr * gr
        want = -lr / (1 - b1 ** step) * m / (torch.sqrt(v / (1 - b2 ** step)) + eps)
        # (a code of the step before is off by its half step, and each step adds another)
        off = (step - 1) * (2.0 ** -4 + 2.0 ** -4 * 1.1) * 1.1 + 1e-5
        moved = p.cpu().double() - before
        assert bool(torch.isfinite(moved).all()), step
        assert bool(((moved - want).abs() <= off * want.abs() + 1e-6 * p.cpu().double().abs()).all()), (
            step, float(((moved - want) / want).abs().max()))
        g.zero_()


def test_adamw_plan_holds_the_memory_of_its_tensors(km):  # noqa: F811
    """A tensor that is given other memory leaves the plan with the old one, which no one else is given."""
    n = 1 << 20
    p, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
    M, V, scales = km.adamw_states([p], 8)
    w = torch.ones(n, device="cuda")
    h = torch.ones(n, device="cuda", dtype=BF16)
    M2, V2, scales2 = km.adamw_states([h], 8)
    km.adamw_plan([p], [g], M, V, scales=scales)  # (dropped at once: holds nothing)
    base = torch.cuda.memory_allocated()
    plans = [km.adamw_plan([p], [g], M, V, scales=scales), km.adamw_plan([h], [g], M2, V2, scales=scales2, masters=[w])]
    tables = torch.cuda.memory_allocated() - base
    for t in (p, g, w, h, *M, *V, *M2, *V2, *scales[0], *scales[1], *scales2[0], *scales2[1]):
        t.data = torch.empty(0, dtype=t.dtype, device="cuda")
    assert torch.cuda.memory_allocated() == base + tables
    del plans
    assert torch.cuda.memory_allocated() < base - 17 * n
