"""AdamW states in 8 bits, rounded stochastically, on the GPU.

One step: each code is one of the two next to the value, and the mean over T step numbers (the averages before their rounding
do not depend on it) is off by a Bernoulli mean's error: with
step h, P(|mean - value| > 3.5 h / sqrt(T)) <= 2 exp(-2 * 3.5^2) = 5e-11 a value; rounding in 32 bits adds 16 u of the value,
the random bits 2^-19 h, and the least code of a positive v has no second one below it.

Runs of steps, against the averages in 64 bits that are never taken from the codes.  A step rounds a value x that was a code
before and moved by d: variance at most h |d|.  With h <= x / 4 (e5m2), E|d| <= (1 - b2) (x + g^2) + x |change of the
block's scale| <= 4 (1 - b2) x, the relative variance of v grows by at most (1 - b2) = 1e-3 a step and stays below 2 over 2,000
steps, whatever v does meanwhile.  A mean of v's ratio over n independent elements is 1 to within five times sqrt(2 / n).
For m: h <= |x| / 8 and an error of at most h / 2 a step, of which 1 / (1 - b1^2) are left (b1 = 0.9: 5.3); errors are
independent of m, so that the coefficient of m8 on m, sum m8 m / sum m^2, is 1 to within five times
sqrt(5.3) / 16 sqrt(sum m^4) / sum m^2 < 1 / sqrt(n) (a normal m's fourth moment is 3).  For b1 = 0.99 an error is a step's
remainder: variance at most h |d| <= x^2 / 8 * 2 * (1 - b1), of which 1 / (1 - b1^2) are left: x^2 / 8.
"""

import math

import pytest
import torch

from tests import test_gpu_train as H
from tests.test_gpu_train import BF16, F16, F32, U, km  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

RATES = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0)


def spacing(x, scale, mant, emin):
    """The distance of the codes next to x, in x's own unit (64 bits)."""
    y = (x.abs() / scale).clamp(min=2.0 ** -40)
    return 2.0 ** (torch.floor(torch.log2(y)).clamp(min=emin) - mant) * scale


def wide(scale, n):
    return scale.double().cpu().repeat_interleave(H.BLOCK)[:n]


def a_state(seed, n, spread=2.0):
    g = H.gen(seed)
    size = torch.exp(torch.randn(n, generator=g) * spread)
    return size * torch.randn(n, generator=g), 0.3 * size * torch.randn(n, generator=g), size.square() * torch.rand(n, generator=g)


def set_states(km, M, V, scales, m, v):  # noqa: F811
    """8-bit states that hold m and v (to nearest)."""
    for t, s, x, top, dt in ((M, scales[0], m, 256.0, torch.float8_e4m3fn), (V, scales[1], v, 32768.0, torch.float8_e5m2)):
        n = x.numel()
        b = torch.nn.functional.pad(x, (0, -n % H.BLOCK)).view(-1, H.BLOCK)
        f = b.abs().amax(-1) / top
        t.view(torch.uint8).copy_((b / f[:, None]).to(dt).view(torch.uint8).view(-1)[:n])
        s.copy_(f)


def test_each_code_is_a_neighbour_and_their_mean_the_value(km):  # noqa: F811
    n, T = 3000, 1500
    g, m, v = a_state(1, n)
    p, G = torch.zeros(n, device="cuda"), g.cuda()
    M, V, scales = km.adamw_states([p], 8)
    plan = km.adamw_plan([p], [G], M, V, scales=scales)
    set_states(km, M[0], V[0], [s[0] for s in scales], m, v)
    keep = [t.view(torch.uint8).clone() for t in (M[0], V[0])], [s[0].clone() for s in scales]
    m0, v0 = H.decoded(M[0], scales[0][0]), H.decoded(V[0], scales[1][0])
    (_, m1, v1), _ = H.adamw_ref(torch.zeros(n), g, m0, v0, 1, **RATES)
    sums = [torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2)]
    lo, hi = [s + math.inf for s in sums], [s - math.inf for s in sums]
    for step in range(1, T + 1):
        for t, old in zip((M[0], V[0], scales[0][0], scales[1][0]), (*keep[0], *keep[1])):
            (t.view(torch.uint8) if t.element_size() == 1 else t).copy_(old)
        km.adamw(plan, step=step, rounding="stochastic", **RATES)
        for k, (t, s) in enumerate(((M[0], scales[0][0]), (V[0], scales[1][0]))):
            x = t.float().double() * s.double().repeat_interleave(H.BLOCK)[:n]
            sums[k] += x
            lo[k], hi[k] = torch.minimum(lo[k], x), torch.maximum(hi[k], x)
    for k, (want, top, mant, emin) in enumerate(((m1, 256.0, 3, -6), (v1, 32768.0, 2, -14))):
        s = wide(scales[k][0], n)
        b = torch.nn.functional.pad(want, (0, -n % H.BLOCK)).view(-1, H.BLOCK)
        high = b.abs().amax(-1)
        H.near(scales[k][0], high / top, 16 * U * high / top, "scale")
        h = spacing(want, s, mant, emin)
        near = 16 * U * want.abs()
        a, z = lo[k].cpu(), hi[k].cpu()
        least = (want > 0) & (want < s * 2.0 ** -16) if k else torch.zeros(n, dtype=torch.bool)
        assert bool((a[least] == z[least]).all()) and (k == 0 or bool((a > 0).all()))
        ok = ~least
        # (T steps need not show both codes: one that is taken with probability q is missing in all of them with (1 - q)^T)
        assert bool((z - a <= h * (1 + 2.0 ** -20))[ok].all())
        assert bool((a >= want - h - near)[ok].all()) and bool((z <= want + h + near)[ok].all())
        assert int((z > a)[ok].sum()) > n // 2
        biggest = want.abs() == high.repeat_interleave(H.BLOCK)[:n]
        assert int(biggest.sum()) == -(-n // H.BLOCK)
        assert bool((a == z)[biggest].all()) and bool(((a - want).abs() <= 16 * U * want.abs())[biggest].all())
        off = (sums[k].cpu() / T - want).abs()[ok]
        assert bool((off <= (3.5 * h / math.sqrt(T) + h * 2.0 ** -19 + near)[ok]).all()), float((off / h[ok]).max() * math.sqrt(T))


def run(km, n, g, steps, offset=0, stream=None):  # noqa: F811
    made = lambda dt: torch.zeros(n + offset, dtype=dt, device="cuda")[offset:]  # noqa: E731
    p, G = made(F32), made(F32)
    G.copy_(g)
    M, V, scales = km.adamw_states([p], 8)
    if offset:
        M, V = [made(torch.uint8).view(torch.float8_e4m3fn)], [made(torch.uint8).view(torch.float8_e5m2)]
    plan = km.adamw_plan([p], [G], M, V, scales=scales)
    torch.cuda.synchronize()
    for k in steps:
        km.adamw(plan, step=k, rounding="stochastic", stream=stream, **RATES)
    torch.cuda.synchronize()
    return [t.view(torch.uint8).clone() for t in (p, M[0], V[0], scales[0][0], scales[1][0])]


def same(a, b):
    return [torch.equal(x, y) for x, y in zip(a, b)]


def test_a_run_repeats_and_its_steps_do_not(km):  # noqa: F811
    n = 9000
    g = a_state(2, n)[0].cuda()
    a = run(km, n, g, (1, 2, 3))
    assert all(same(a, run(km, n, g, (1, 2, 3))))
    assert all(same(a, run(km, n, g, (1, 2, 3), stream=torch.cuda.Stream())))
    # the same values whatever the arrays' alignment
    assert all(same(a, run(km, n, g, (1, 2, 3), offset=1)))
    one, two = run(km, n, g, (5,)), run(km, n, g, (6,))
    assert not any(same(one, two)[1:3])
    assert all(same(one, two)[3:])  # (from zero states: the same values, other codes)


def test_captured_steps_are_the_eager_ones(km):  # noqa: F811
    n = 5000
    g = a_state(3, n)[0].cuda()
    def fresh():
        p = torch.zeros(n, device="cuda")
        M, V, s = km.adamw_states([p], 8)
        return km.adamw_plan([p], [g], M, V, scales=s), [p, M[0], V[0], s[0][0], s[1][0]]
    a, b = fresh(), fresh()
    step, lr = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.tensor([1e-3], device="cuda")
    rates = {**RATES, "lr": lr}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        km.adamw(a[0], step=step, rounding="stochastic", **rates)
    for k in range(1, 5):
        graph.replay()
        torch.cuda.synchronize()
        km.adamw(b[0], step=torch.tensor([k], device="cuda"), rounding="stochastic", **rates)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[1], b[1])), k


def test_nan_infinities_and_zeros(km):  # noqa: F811
    n = 1000
    p, g = torch.ones(n, device="cuda"), torch.full((n,), 0.5, device="cuda")
    g[7], g[300], g[301], g[600], g[601:] = math.nan, math.inf, 0.0, 1e25, 0.0
    M, V, scales = km.adamw_states([p], 8)
    plan = km.adamw_plan([p], [g], M, V, scales=scales)
    km.adamw(plan, step=1, rounding="stochastic", **RATES)
    m, v = M[0].float().cpu(), V[0].float().cpu()
    fin = torch.ones(n, dtype=torch.bool)
    fin[[7, 300]] = False
    assert bool(torch.isfinite(m)[fin].all()) and bool(torch.isnan(m)[~fin].all())
    assert bool(torch.isnan(v[7])) and float(v[300]) == math.inf and float(v[600]) == math.inf
    fin[600] = False
    assert bool(torch.isfinite(v)[fin].all()) and bool(torch.isfinite(p.cpu())[torch.arange(n) != 7][:290].all())
    assert not m[768:].any() and not v[768:].any() and bool((v[768:] == 0).all())
    assert not m[301] and not v[301]


def averages(km, betas, change, steps, blocks=64, seed=0):  # noqa: F811
    """m and v held in 8 bits after `steps` steps beside the averages in 64 bits; change(k, gradients) sets a step's."""
    n = blocks * H.BLOCK
    gpu = torch.Generator(device="cuda")
    gpu.manual_seed(seed)
    size = torch.exp(torch.randn(n, generator=gpu, device="cuda"))
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    M, V, scales = km.adamw_states([p], 8)
    plan = km.adamw_plan([p], [g], M, V, scales=scales)
    m, v = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    b1, b2 = betas
    for k in range(1, steps + 1):
        torch.randn(n, generator=gpu, device="cuda", out=g)
        g.mul_(size)
        change(k, g)
        km.adamw(plan, step=k, rounding="stochastic", **{**RATES, "betas": betas})
        m.mul_(b1).add_(g, alpha=1 - b1)
        v.mul_(b2).add_(g.double().square(), alpha=1 - b2)
    factor = [s[0].double().repeat_interleave(H.BLOCK) for s in scales]
    return M[0].float().double() * factor[0], m, V[0].float().double() * factor[1], v


def coefficient(a, b):
    return float((a * b).sum() / (b * b).sum())


def fall(to):
    def change(k, g):
        if k > 1000:
            g.view(-1, 2)[:, 0] *= to
    return change


def spike(k, g):
    if k == 1000:
        g.view(-1, H.BLOCK)[:, 0] *= 300


@pytest.mark.parametrize("change", [fall(0.1), fall(0.0), spike, lambda k, g: None], ids=["fall", "stop", "spike", "steady"])
@pytest.mark.parametrize("steps", [1000, 2000, 3000])
def test_v_follows_its_average(km, change, steps):  # noqa: F811
    _, _, v8, v = averages(km, (0.9, 0.999), change, steps)
    for half in (slice(0, None, 2), slice(1, None, 2)):
        ratio = v8[half] / v[half]
        assert abs(float(ratio.mean()) - 1) <= 5 * math.sqrt(2 / ratio.numel()), float(ratio.mean())


@pytest.mark.parametrize("b1", [0.9, 0.99])
def test_m_follows_its_average(km, b1):  # noqa: F811
    # (a gradient with a mean of its own, whose sign turns at step 1,000)
    def drift(k, g):
        g.mul_(0.5).add_(torch.sign(torch.arange(g.numel(), device="cuda") % 2 - 0.5), alpha=1.0 if k <= 1000 else -1.0)
    m8, m, _, _ = averages(km, (b1, 0.999), drift, 1500)
    assert abs(coefficient(m8, m) - 1) <= 5 / math.sqrt(m.numel()), coefficient(m8, m)


def test_no_rounding_of_states_in_32_bits(km):  # noqa: F811
    p, g = torch.ones(5, device="cuda"), torch.ones(5, device="cuda")
    M, V, scales = km.adamw_states([p])
    plan = km.adamw_plan([p], [g], M, V)
    for kw in (dict(rounding="stochastic"), dict(rounding="up"), dict(rounding=None)):
        with pytest.raises(km.KMeansError):
            km.adamw(plan, lr=0.1, step=1, **kw)
    assert bool((p == 1).all())


@pytest.mark.parametrize("pdt, gdt, masters", [(F32, F32, False), (BF16, BF16, True), (F16, F32, True), (BF16, F16, False)])
@pytest.mark.parametrize("each", [[1], [255, 256, 257], [4095, 1, 4097, 0, 12288, 3], [9_000_001]])
def test_types_and_sizes(km, each, pdt, gdt, masters):  # noqa: F811
    """From zero states: the parameters as with states in 32 bits (codes are not in the step), each code a neighbour."""
    g = H.gen(len(each))
    W = [torch.randn(n, generator=g) for n in each]
    P = [w.to(pdt).cuda() for w in W]
    G = [torch.randn(n, generator=g).to(gdt).cuda() for n in each]
    copies = [w.cuda() for w in W] if masters else None
    M, V, scales = km.adamw_states(P, 8)
    plan = km.adamw_plan(P, G, M, V, scales=scales, masters=copies)
    start = [w.clone() if masters else p.cpu() for w, p in zip(W, P)]
    km.adamw(plan, step=1, rounding="stochastic", **H.RATES)
    for i, n in enumerate(each):
        (p, m, v), (tp, tm, tv) = H.adamw_ref(start[i], G[i].cpu(), torch.zeros(n), torch.zeros(n), 1, **H.RATES)
        if masters:
            H.near(copies[i], p, tp, "master")
            assert torch.equal(P[i].cpu(), copies[i].cpu().to(pdt))
        else:
            H.near(P[i], p, tp + H.half_step(pdt) * (p.abs() + tp) * (pdt != F32) + H.tiny(pdt), "p")
        for t, s, want, tol, mant, emin in ((M, scales[0], m, tm, 3, -6), (V, scales[1], v, tv, 2, -14)):
            f = wide(s[i], n)
            h = spacing(want, f, mant, emin)
            bound = h * (1 + 2.0 ** -20) + tol + 16 * U * want.abs()
            H.near(H.decoded(t[i], s[i]), want, bound, "state")
