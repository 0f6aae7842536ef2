"""The paths of the training operators behind the first ones: many rows (whole registers a lane, waves that loop), mass
ties and near-ties there, long rows, wide tiles of the gradient, steps that are streamed.  References are in 64 bits, on
the GPU where they are large; tolerances as in test_gpu_train."""

import math

import pytest
import torch

from tests import test_gpu_train as H
from tests.test_gpu_train import BF16, F16, F32, TYPES, check_route, check_route_grad, gen, some_bias, some_logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_means_clustering_amd as km
    return km


def many(K, rows=None):
    """Rows enough for the kernels of many rows (2^21 choices), no round number."""
    return rows or (1 << 21) // K + 77


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K, S", [(17, 3), (32, 8), (32, 20), (50, 2), (64, 6), (100, 8), (128, 8), (128, 10), (160, 1),
                                  (256, 8), (256, 32), (300, 8), (512, 2), (512, 16)])
def test_route_of_many_rows(km, dtype, K, S):
    n = many(K)
    x = some_logits(n, K, dtype, K + S).cuda()
    b = some_bias(K, K).cuda()
    for kw in (dict(), dict(renormalise=False), dict(score="sigmoid", scale=2.0), dict(bias=b), dict(bias=b, score="sigmoid"),
               dict(bias=b, renormalise=False)):
        check_route(km.route(x, S, **kw), x, S, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K, groups, top_groups, S", [(32, 32, 5, 4), (32, 4, 2, 8), (60, 6, 2, 7), (64, 8, 3, 8),
                                                      (160, 8, 3, 6), (256, 8, 4, 8), (256, 64, 20, 16), (252, 7, 3, 8),
                                                      (512, 16, 4, 8)])
def test_route_of_many_rows_in_groups(km, dtype, K, groups, top_groups, S):
    x = some_logits(many(K), K, dtype, K + groups).cuda()
    b = some_bias(K, K).cuda()
    for score in ("softmax", "sigmoid"):
        for bias in (None, b):
            for best in (1, 2):
                kw = dict(score=score, bias=bias, groups=groups, top_groups=top_groups, group_best=best)
                check_route(km.route(x, S, **kw), x, S, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [24, 64, 256])
def test_route_of_many_rows_with_ties_and_choices_out(km, dtype, K):
    n = many(K)
    g = gen(K)
    x = torch.randint(0, 4, (n, K), generator=g).to(dtype)
    x[torch.rand(n, K, generator=g) < 0.3] = -math.inf
    x[5] = -math.inf
    x[6], x[7, 3] = math.nan, math.nan
    x[8, 4] = math.inf
    valid = torch.rand(n, generator=g) < 0.9
    valid[5:9] = True
    x[~valid] = math.nan
    y = torch.where(valid[:, None], x, 0.0).to(dtype).cuda()
    x, valid = x.cuda(), valid.cuda()
    off = some_bias(K, 3).cuda()
    off[K // 3], off[0] = -math.inf, math.inf
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(K, device="cuda"), off):
            for groups in (1, 4):
                kw = dict(score=score, bias=bias, groups=groups, top_groups=2 if groups > 1 else 1, valid=valid)
                check_route(km.route(x, 6, **kw), y, 6, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("K, S", [(32, 4), (128, 8), (512, 8)])
def test_route_of_many_rows_of_neighbouring_scores(km, score, K, S):
    n = many(K)
    x = torch.randn(n, K, generator=gen(K)).cuda()
    h = K // 2
    x[:, h:] = torch.nextafter(x[:, :h], torch.full((), math.inf, device="cuda"))
    for bias in (torch.zeros(K, device="cuda"), torch.full((K,), 0.125, device="cuda")):
        for groups in (1, 4):
            kw = dict(score=score, bias=bias, groups=groups, top_groups=2 if groups > 1 else 1)
            check_route(km.route(x, S, **kw), x, S, **kw)
    # every score nearly the same
    near = (0.7 - H.scores(x[0].double(), score)).float()
    y = x[:1].repeat(n, 1)
    for groups in (1, 4):
        kw = dict(score=score, bias=near, groups=groups, top_groups=3 if groups > 1 else 1)
        check_route(km.route(y, S, **kw), y, S, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_waves_that_loop(km, dtype):
    # more tiles than waves, of plain rows and of scored ones
    for n, K, S, kw in ((140_003, 256, 8, dict()), (140_003, 256, 2, dict(renormalise=False)),
                        (60_011, 256, 8, dict(bias=some_bias(256, 1).cuda(), score="sigmoid", groups=8, top_groups=4)),
                        (2_100_003, 8, 2, dict())):
        g = torch.Generator(device="cuda")
        g.manual_seed(n)
        x = torch.randn(n, K, generator=g, device="cuda").to(dtype)
        valid = torch.rand(n, generator=g, device="cuda") < 0.95
        kw = dict(kw, valid=valid)
        check_route(km.route(x, S, **kw), x, S, **kw)


def test_route_at_odd_addresses_of_many_rows(km):
    for dt in TYPES:
        for K in (33, 100, 511):
            n = many(K)
            x = some_logits(n, K, dt, K).cuda()
            buf = torch.full((3 + n * K + 9,), math.nan, dtype=dt, device="cuda")
            buf[3:3 + n * K] = x.view(-1)
            y = buf[3:3 + n * K].view(n, K)
            b = some_bias(K, 1).cuda()
            check_route(km.route(y, 5), x, 5)
            check_route(km.route(y, 5, bias=b), x, 5, bias=b)


@pytest.mark.parametrize("K, S", [(2049, 2), (4096, 8), (10007, 20), (70000, 8)])
def test_route_of_long_rows(km, K, S):
    for dt in TYPES:
        x = some_logits(9, K, dt, K)
        x[1, :2048] = -math.inf
        x[2, 2048:] = -math.inf
        x[3] = 1.0
        for kw in (dict(), dict(renormalise=False), dict(score="sigmoid")):
            check_route(km.route(x.cuda(), S, **kw), x, S, **kw)
    if K < 20000:
        x = some_logits(4, K, F32, K)
        b = some_bias(K, 1)
        check_route(km.route(x.cuda(), S, bias=b.cuda(), score="sigmoid"), x, S, bias=b, score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n, K, S", [(9, 8, 2), (9, 60, 4), (2_300, 1000, 8), (17, 256, 12), (5_000, 511, 5), (3, 2048, 32)])
def test_route_of_copies_behind_the_selection(km, score, n, K, S):
    """Equal choices at a row's end that 32 bits do not tell from lower ones in front of them, and that belong to the
    selection: two of them, as many as there are selections, and more."""
    x = torch.full((n, K), -9.0) - torch.rand(n, K, generator=gen(K))
    b = torch.zeros(K)
    low, high = torch.tensor(-5.0), torch.nextafter(torch.tensor(-5.0), torch.tensor(0.0))
    b[: K // 2], b[K // 2:] = 1.0, 1.0
    for i in range(n):
        copies = (2, S, S + 2)[i % 3]
        x[i, 1:1 + S] = low
        x[i, K - copies:] = high
        if i % 2:
            x[i, 0] = 2.0
    check_route(km.route(x.cuda(), S, score=score, bias=b.cuda()), x, S, score=score, bias=b)


@pytest.mark.parametrize("K", [12, 64, 320, 2304])
def test_route_of_extreme_biases(km, K):
    """Biases that absorb the scores (ties then go to the lowest index), whose sums pass fp32, and that force choices in
    and out."""
    x = some_logits(40, K, F32, K)
    x[1] = -math.inf
    x[2, : K // 2] = -math.inf
    kinds = torch.tensor([3e38, 3e38, -3e38, 1e30, 0.0, 0.001, -0.002, math.inf, -math.inf])
    for seed, some in enumerate((slice(0, 7), slice(0, 9), slice(3, 6), slice(7, 9), slice(2, 3))):
        of = kinds[some]
        b = of[torch.randint(0, len(of), (K,), generator=gen(seed))]
        for score in ("softmax", "sigmoid"):
            for kw in (dict(), dict(groups=4, top_groups=2), dict(groups=4, top_groups=3, group_best=1)):
                kw = dict(score=score, bias=b, **kw)
                check_route(km.route(x.cuda(), 5, **{**kw, "bias": b.cuda()}), x, 5, **kw)


@pytest.mark.parametrize("K, groups, S", [(8192, 1, 64), (8192, 64, 33), (8193, 3, 9), (2052, 4, 3), (40, 5, 36), (1, 1, 1)])
def test_route_of_rows_taken_in_64_bits(km, K, groups, S):
    """Rows with scores that are too long for a wave's registers, and more selections than its lists, or than a lane's
    best; with equal scores, choices that are out and rows without any."""
    n = 37
    x = some_logits(n, K, F32, K)
    x[1] = -math.inf
    x[2, : K - K // 3] = -math.inf
    x[3] = 0.25
    x[4, ::2] = x[4, 0]
    b = some_bias(K, 1)
    valid = torch.ones(n, dtype=torch.bool)
    valid[5] = False
    for score in ("softmax", "sigmoid"):
        kw = dict(score=score, groups=groups, top_groups=(groups + 1) // 2)
        if S * groups > K * kw["top_groups"]:
            kw["top_groups"] = groups
        check_route(km.route(x.cuda(), S, bias=b.cuda(), valid=valid.cuda(), **kw), x, S, bias=b, valid=valid, **kw)
        check_route(km.route(x.cuda(), S, renormalise=False, **kw), x, S, renormalise=False, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, K, S", [(30_001, 64, 8), (9_001, 256, 5), (70_001, 8, 2), (3_001, 1024, 2), (2_001, 2048, 3),
                                     (20_011, 100, 64), (333, 4100, 7), (65, 20_000, 16)])
def test_route_grad_of_many_rows(km, dtype, n, K, S):
    x = some_logits(n, K, dtype, n).cuda()
    g = gen(n)
    valid = (torch.rand(n, generator=g) < 0.9).cuda()
    ids, _, z = km.route(x, S, valid=valid)
    dw = torch.randn(n, S, generator=g).cuda()
    old = torch.randn(n, K, generator=g).to(dtype).cuda()
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            kw = dict(score=score, renormalise=renormalise, scale=1.5)
            check_route_grad(km.route_grad(x, ids, z, dw, **kw), x, ids, dw, **kw)
            out = old.clone()
            km.route_grad(x, ids, z, dw, out=out, accumulate=True, **kw)
            check_route_grad(out, x, ids, dw, old=old, **kw)
            assert torch.equal(out[~valid], old[~valid])


def test_route_grad_of_the_same_id_in_whole_rows(km):
    # repeated ids where a team holds the row: sums in the order of the selections, and the LDS clean for the next rows
    g = gen(4)
    for K in (8, 16, 40, 128, 1000, 2048):
        n = 5000 if K < 1000 else 300
        x = some_logits(n, K, F32, K, spread=1.0).cuda()
        ids = torch.randint(0, 3, (n, 8), generator=g).to(torch.int32).cuda()
        ids[::3, 4:] = -1
        ids[1::3] = torch.arange(8, dtype=torch.int32, device="cuda") % K
        dw = torch.randn(n, 8, generator=g).cuda()
        z = x.gather(1, ids.long().clamp(min=0))
        got = km.route_grad(x, ids, z, dw, renormalise=False)
        check_route_grad(got, x, ids, dw, renormalise=False)
        assert torch.equal(got, km.route_grad(x, ids, z, dw, renormalise=False))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt, gdt, masters", [(F32, F32, False), (BF16, BF16, True), (F16, F32, True)])
def test_adamw_streamed(km, bits, pdt, gdt, masters):
    # more than 128 MiB moved; the tensors' ends and a small one among them
    g = torch.Generator(device="cuda")
    g.manual_seed(bits)
    each = [9_000_001, 4097, 1_000_000]
    W = [torch.randn(n, generator=g, device="cuda") for n in each]
    P = [w.to(pdt) for w in W] if masters else [w.to(pdt) for w in W]
    G = [torch.randn(n, generator=g, device="cuda").to(gdt) for n in each]
    M, V, scales = km.adamw_states(P, bits)
    plan = km.adamw_plan(P, G, M, V, scales=scales, masters=W if masters else None)
    start = [(w if masters else p).clone() for w, p in zip(W, P)]
    km.adamw(plan, step=1, **H.RATES)
    for i in range(3):
        zero = torch.zeros_like(G[i], dtype=F32)
        (p, m, v), (tp, tm, tv) = H.adamw_ref(start[i], G[i], zero, zero, 1, **H.RATES)
        got = (W[i] if masters else P[i]).double()
        tol = tp if masters or pdt == F32 else tp + H.half_step(pdt) * (p.abs() + tp) + H.tiny(pdt)
        assert bool(((got - p).abs() <= tol).all())
        if masters:
            assert torch.equal(P[i], W[i].to(pdt))
        if bits == 32:
            assert bool(((M[i].double() - m).abs() <= tm).all()) and bool(((V[i].double() - v).abs() <= tv).all())
        else:
            H.check_8bit(M[i], scales[0][i], m.cpu(), tm.cpu(), 256.0, 2.0 ** -4, 2.0 ** -10, "m")
            H.check_8bit(V[i], scales[1][i], v.cpu(), tv.cpu(), 32768.0, 2.0 ** -3, 2.0 ** -16, "v")


def test_adamw_plans_share_nothing(km):
    """Two plans over the same tensors, stepped in turn, are one plan stepped twice."""
    def fresh():
        p = torch.linspace(-1, 1, 5000, device="cuda")
        g = torch.linspace(2, -3, 5000, device="cuda")
        M, V, s = km.adamw_states([p], 8)
        return p, [km.adamw_plan([p], [g], M, V, scales=s) for _ in range(2)]
    (p, a), (q, b) = fresh(), fresh()
    for k in (1, 2):
        km.adamw(a[0], step=k, **H.RATES)
        km.adamw(b[k - 1], step=k, **H.RATES)
    assert torch.equal(p, q)

