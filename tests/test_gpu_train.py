"""The training operators on the GPU against their definitions in 64 bits.

Tolerances count roundings (u = 2^-24, half a step of fp32; half a step of the output's type is eps / 2):
  route       ids, and chosen, are exact.  With R the largest distance of a logit from the one that the row's exponentials
              are taken relative to (at most 104: exp of less is 0 in fp32), an exponential is off by (R + 4) u relative
              (the difference's rounding, its scaling, exp itself), a score by 4 u more (1 + e, the quotient), a sum of the
              row's K values by K / 64 + 40 u (lanes add 32 values one after another and K / 64 where rows are longer, then
              pairs), a sum of S shares by S u; two such numbers meet in a quotient, and two products follow.
  route_grad  w as above; the mean of the dweights under w by that and S u of its magnitude; the difference, the products
              and the output's type add 4 u and half a step; a row's sum of p * dweights, where every choice has one, by
              another K / 64 + 40.
  adamw       m and v: three roundings of each term and one of the sum; the step: 4 u for the root, its factor, eps, 3 u
              for the quotient and the rate; the parameter: 3 u.  In 8 bits the codes add half a step of their format.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]


@pytest.fixture(scope="module")
def km():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import exact_means_clustering_amd as km
    return km


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the smallest positive value's step (fp32 results may also be flushed below its normal range)."""
    return {F32: 2.0 ** -126, F16: 2.0 ** -25, BF16: 2.0 ** -126}[dtype]


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


# ---- routing: the definition ------------------------------------------------------------------------------------------

def scores(x, score):
    return torch.softmax(x, -1) if score == "softmax" else 1.0 / (1.0 + torch.exp(-x))


def route_ref(x, S, score="softmax", bias=None, groups=1, top_groups=None, group_best=2, renormalise=True, scale=1.0,
              valid=None, tilt=0.0):
    """ids, weights, chosen of logits [N, K], in 64 bits; tilt: added to a group's worth for each index it comes earlier."""
    n, K = x.shape
    x = x.double()
    top_groups = groups if top_groups is None else top_groups
    arith = bias is not None or (groups > 1 and top_groups < groups and group_best == 2 and K > groups)
    s = scores(x, score)
    bad = torch.isnan(x).any(-1) | ((x == math.inf).any(-1) if score == "softmax" else False)
    if bias is not None:
        bad = bad | torch.isnan(bias).any()
    c = s + (0.0 if bias is None else bias.double()) if arith else x.clone()
    c[x == -math.inf] = -math.inf
    c = torch.nan_to_num(c, nan=0.0, posinf=math.inf, neginf=-math.inf)
    if top_groups < groups:
        per = c.view(n, groups, K // groups)
        best = torch.sort(per, dim=-1, descending=True).values[..., :min(group_best, K // groups)]
        worth = torch.where(best > -math.inf, best, 0.0).sum(-1)
        worth = worth - tilt * torch.arange(groups, device=x.device)
        worth[best[..., 0] == -math.inf] = -math.inf
        order = torch.sort(worth, dim=-1, descending=True, stable=True).indices[:, :top_groups]
        keep = torch.zeros(n, groups, dtype=torch.bool, device=x.device).scatter_(1, order, True)
        c = torch.where(keep[..., None], per, -math.inf).view(n, K)
    top, ids = torch.sort(c, dim=-1, descending=True, stable=True)
    ids, live = ids[:, :S].clone(), (top[:, :S] > -math.inf) & ~bad[:, None]
    if valid is not None:
        live &= valid[:, None]
        bad = bad & valid
    z = torch.where(live, x.gather(1, ids), -math.inf)
    ids[~live] = -1
    w, _ = weights_ref(x, ids, z, score, renormalise)
    w = w * scale
    w[bad], z[bad] = math.nan, math.nan
    return ids.to(torch.int32), w, z


def weights_ref(x, ids, z, score, renormalise):
    """(weights, R) of ids [N, S] with logits z, before the scale."""
    live = ids >= 0
    high = z.amax(-1, keepdim=True)
    if not renormalise and score == "softmax":
        high = torch.where(torch.isfinite(x), x, -math.inf).amax(-1, keepdim=True)
    high = torch.where(torch.isfinite(high), high, 0.0)
    R = torch.where(torch.isfinite(z), (high - z).abs().clamp(max=104), 0.0).amax(-1, keepdim=True)
    if score == "sigmoid":
        R = torch.where(torch.isfinite(z), z.abs().clamp(max=104), 0.0).amax(-1, keepdim=True).maximum(R)
    if renormalise:
        if score == "softmax":
            e = torch.exp(torch.where(live, z - high, -math.inf))
        else:  # log sigmoid, relative to the row's largest
            ls = torch.where(live, torch.nn.functional.logsigmoid(z), -math.inf)
            e = torch.exp(ls - torch.where(live.any(-1, keepdim=True), ls.amax(-1, keepdim=True), 0.0))
        w = torch.where(live, e / e.sum(-1, keepdim=True), 0.0)
    else:
        s = torch.softmax(torch.where(x == -math.inf, -1e30, torch.nan_to_num(x)), -1) if score == "softmax" else scores(
            x, score)
        w = torch.where(live, s.gather(1, ids.long().clamp(min=0)), 0.0)
    return w, R


def rel_of(R, K, S):
    return (2 * R + 2 * 4 + 2 * 4 + K / 64 + 40 + S + 4) * U * 1.01


def check_route(got, x, S, **kw):
    ids, w, z = (t.to(x.device) for t in got)
    rid, rw, rz = route_ref(x, S, **kw)
    assert ids.dtype == torch.int32 and w.dtype == F32 and z.dtype == F32
    if kw.get("groups", 1) > 1 and kw.get("bias") is not None:
        # Worths are sums (s + b) + (s' + b') of biases that are multiples of a thousandth: two of them may be equal in
        # exact arithmetic (0.011 + 0.032 and 0.034 + 0.009 beside the same s) and differ in the last bit of 64, with the
        # last bit of s.  A 64-bit worth below 4 is off by at most 8 2^-53 < 2^-49: such rows may go either way.
        for tilt in (2.0 ** -48, -(2.0 ** -48)):
            other = route_ref(x, S, **kw, tilt=tilt)
            take = (ids.view(rid.shape) != rid).any(-1) & (ids.view(rid.shape) == other[0]).all(-1)
            rid, rw, rz = (torch.where(take[:, None], b, a) for a, b in zip((rid, rw, rz), other))
    bad = (ids.view(rid.shape) != rid).any(-1).nonzero()[:, 0]
    assert bad.numel() == 0, (bad.numel(), int(bad[0]), ids.view(rid.shape)[bad[0]], rid[bad[0]])
    assert torch.equal(torch.nan_to_num(z.view(rz.shape).double(), nan=7e77), torch.nan_to_num(rz, nan=7e77))
    _, R = weights_ref(x.double(), rid, torch.nan_to_num(rz, nan=-math.inf), kw.get("score", "softmax"),
                       kw.get("renormalise", True))
    w = w.view(rw.shape).double()
    assert torch.equal(torch.isnan(w), torch.isnan(rw))
    tol = rel_of(R, x.shape[1], S) * rw.abs() + 2.0 ** -126 * kw.get("scale", 1.0)
    off = torch.nan_to_num((w - rw).abs() / tol)
    assert float(off.max() if off.numel() else 0) <= 1, float(off.max())


def some_logits(n, K, dtype, seed, spread=1.5):
    g = gen(seed)
    return (torch.randn(n, K, generator=g) * spread + torch.randn(1, K, generator=g)).to(dtype)


def some_bias(K, seed, steps=40):
    return torch.randint(-steps, steps + 1, (K,), generator=gen(seed)).float() * 0.001


# one row and many, one choice and long rows, every number of lanes a row, odd lengths, all choices selected
ROUTE_SHAPES = [(1, 1, 1), (5, 3, 2), (300, 8, 2), (64, 8, 8), (130, 7, 3), (17, 16, 4), (40, 15, 9), (33, 20, 20), (70, 32, 8),
                (19, 33, 1), (100, 64, 6), (9, 128, 8), (257, 128, 8), (50, 160, 6), (12, 160, 40), (31, 256, 8), (8, 256, 32),
                (3, 300, 33), (6, 512, 16), (5, 1000, 2), (4, 2048, 8), (3, 2049, 8), (2, 5000, 64), (2, 8200, 10),
                (1025, 96, 10)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, K, S", ROUTE_SHAPES)
def test_route(km, dtype, n, K, S):
    x = some_logits(n, K, dtype, n + K)
    for score in ("softmax", "sigmoid"):
        for bias in (None, some_bias(K, K)):
            for renormalise in (True, False):
                kw = dict(score=score, bias=bias, renormalise=renormalise, scale=2.5 if bias is not None else 1.0)
                got = km.route(x.cuda(), S, **{**kw, "bias": cuda(bias)[0]})
                assert got[0].shape == got[1].shape == got[2].shape == (n, S)
                check_route(got, x, S, **kw)


GROUPS = [(8, 4, 2, 2), (8, 2, 1, 3), (20, 5, 3, 6), (64, 64, 9, 8), (64, 32, 5, 8), (64, 2, 1, 16), (160, 8, 3, 6), (256, 8, 4, 8),
          (256, 16, 2, 32), (144, 9, 4, 8), (33, 11, 2, 5), (300, 3, 2, 40), (512, 64, 7, 12), (2048, 32, 5, 8),
          (2112, 33, 4, 8), (4160, 8, 2, 6), (30, 30, 12, 12)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K, groups, top_groups, S", GROUPS)
def test_route_of_groups(km, dtype, K, groups, top_groups, S):
    n = 70 if K < 1000 else 5
    x = some_logits(n, K, dtype, K + groups)
    for score in ("softmax", "sigmoid"):
        for bias in (None, some_bias(K, K)):
            for best in (1, 2):
                kw = dict(score=score, bias=bias, groups=groups, top_groups=top_groups, group_best=best,
                          renormalise=best == 2, scale=1.5)
                check_route(km.route(x.cuda(), S, **{**kw, "bias": cuda(bias)[0]}), x, S, **kw)


@pytest.mark.parametrize("K, S, groups, top_groups", [(6, 6, 1, 1), (8, 4, 4, 2), (100, 10, 5, 2), (3000, 12, 1, 1)])
@pytest.mark.parametrize("dtype", TYPES)
def test_route_with_choices_out(km, dtype, K, S, groups, top_groups):
    # choices out of use, rows with fewer than S of them, with none; groups with none; rows that are not valid hold anything
    x = some_logits(60, K, dtype, K)
    g = gen(K)
    x[torch.rand(60, K, generator=g) < 0.5] = -math.inf
    x[3] = -math.inf
    x[4, 1:] = -math.inf
    x[5, : K // 2] = -math.inf
    valid = torch.rand(60, generator=g) < 0.8
    valid[3:6] = True
    hidden = x.clone()
    hidden[~valid] = math.nan
    bias = some_bias(K, 3)
    off = bias.clone()
    off[K // 3], off[0] = -math.inf, 5.0
    for score in ("softmax", "sigmoid"):
        for b in (None, bias, off):
            for renormalise in (True, False):
                kw = dict(score=score, bias=b, groups=groups, top_groups=top_groups, renormalise=renormalise, valid=valid)
                got = km.route(hidden.cuda(), S, **{**kw, "bias": cuda(b)[0], "valid": valid.cuda()})
                check_route(got, x, S, **kw)
                assert bool((got[0].cpu()[~valid] == -1).all()) and not got[1].cpu()[~valid].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K, S", [(8, 3), (64, 8), (200, 20), (2500, 8)])
def test_route_ties_go_to_the_lowest_index(km, dtype, K, S):
    g = gen(K)
    x = torch.randint(0, 3, (90, K), generator=g).to(dtype)
    x[0] = 0.0
    x[1] = -0.0
    x[2, ::2] = -0.0
    x[2, 1::2] = 0.0
    bias = torch.randint(-1, 2, (K,), generator=g).float() * 0.25
    for score in ("softmax", "sigmoid"):
        for b in (None, torch.zeros(K), bias):
            for groups in (1, 4):
                # (bias 0.25 and -0.25 make scores meet only where logits do: scores of different logits differ by more)
                kw = dict(score=score, bias=b, groups=groups, top_groups=2 if groups > 1 else 1)
                check_route(km.route(x.cuda(), S, **{**kw, "bias": cuda(b)[0]}), x, S, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("K, S", [(16, 4), (128, 8), (1000, 8)])
def test_route_order_of_neighbouring_scores(km, score, K, S):
    # scores a few roundings of fp32 apart, which 32-bit arithmetic puts in any order; the bias makes them meet
    g = gen(K)
    x = torch.randn(200, K, generator=g)
    n = K // 2
    base = x[:, :n].clone()
    x[:, n:2 * n] = torch.nextafter(base, torch.full_like(base, math.inf))   # next to the first half
    x[::3, n:2 * n] = torch.nextafter(x[::3, n:2 * n], torch.full_like(base[::3], -math.inf))
    bias = torch.zeros(K)
    for b in (None, bias, bias + 0.125):
        kw = dict(score=score, bias=b)
        check_route(km.route(x.cuda(), S, **{**kw, "bias": cuda(b)[0]}), x, S, **kw)
    # biases that undo the difference of two scores up to their last bits
    s = scores(x[0].double(), score)
    y = x[:1].repeat(40, 1)
    near = (0.7 - s).float()
    near[K // 4:] = -3.0
    kw = dict(score=score, bias=near)
    check_route(km.route(y.cuda(), S, score=score, bias=near.cuda()), y, S, **kw)
    if K % 4 == 0:
        kw = dict(score=score, bias=near, groups=4, top_groups=2)
        check_route(km.route(y.cuda(), S, score=score, bias=near.cuda(), groups=4, top_groups=2), y, S, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [5, 64, 1500, 4000])
def test_route_of_extreme_logits(km, dtype, K):
    fi = torch.finfo(dtype)
    x = some_logits(16, K, dtype, K)
    x[0] = fi.min
    x[1, 1:] = fi.min
    x[2, : K // 2] = -math.inf
    x[3] = -math.inf
    x[4, K - 1] = fi.max
    x[5] = fi.max
    x[6, 2] = math.nan
    x[7, 3] = math.inf
    x[8] = math.nan
    x[9] = -80.0
    x[10] = -300.0 - torch.arange(K) % 7
    x[11, 0] = fi.tiny
    x[12] = math.inf
    S = min(4, K)
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            for b in (None, some_bias(K, 2)):
                if b is not None and score == "sigmoid":
                    # (scores that a bias absorbs are not told apart, even in 64 bits: only rows of plain size)
                    rows = [2, 3, 6, 8, 13, 14, 15]
                elif b is not None:
                    rows = [2, 3, 6, 7, 8, 12, 13, 14, 15]
                else:
                    rows = list(range(16))
                kw = dict(score=score, renormalise=renormalise, bias=b)
                check_route(km.route(x[rows].contiguous().cuda(), S, **{**kw, "bias": cuda(b)[0]}), x[rows], S, **kw)


def test_route_of_a_nan_bias(km):
    x = some_logits(9, 40, F32, 1)
    bias = some_bias(40, 1)
    bias[7] = math.nan
    check_route(km.route(x.cuda(), 4, bias=bias.cuda()), x, 4, bias=bias)


@pytest.mark.parametrize("off", [1, 2, 3, 4])
def test_route_at_odd_addresses(km, off):
    for dt in TYPES:
        for K in (5, 16, 24, 40, 200, 2060):
            n = 77 if K < 1000 else 5
            x = some_logits(n, K, dt, off)
            buf = torch.full((off + n * K + 9,), math.nan, dtype=dt, device="cuda")
            buf[off:off + n * K] = x.view(-1).cuda()
            v = torch.zeros(n + off, dtype=torch.bool, device="cuda")[off:]
            v.fill_(True)
            check_route(km.route(buf[off:off + n * K].view(n, K), 5, valid=v), x, 5)
            b = some_bias(K, 1)
            check_route(km.route(buf[off:off + n * K].view(n, K), 5, bias=b.cuda(), score="sigmoid"), x, 5, bias=b,
                        score="sigmoid")


def test_route_offsets_past_32_bits(km):
    n, K = (1 << 21) + 5, 1032                  # 2^31 + elements
    x = torch.zeros(n, K, dtype=BF16, device="cuda")
    x[:, 7], x[:, 9] = 2.0, 1.0
    tail = some_logits(2, K, BF16, 1)
    x[-2:] = tail.cuda()
    got = km.route(x, 2)
    assert bool((got[0][:-2] == torch.tensor([7, 9], device="cuda", dtype=torch.int32)).all())
    check_route([t[-2:] for t in got], tail, 2)
    got = km.route(x, 2, bias=torch.zeros(K, device="cuda"), groups=4, top_groups=3)
    assert bool((got[0][:-2] == torch.tensor([7, 9], device="cuda", dtype=torch.int32)).all())
    check_route([t[-2:] for t in got], tail, 2, bias=torch.zeros(K), groups=4, top_groups=3)
    dw = torch.ones(n, 2, device="cuda")
    dw[:, 1] = 3.0
    dx = km.route_grad(x, got[0], got[2], dw)
    assert not dx[:-2, 10:].any() and bool((dx[:-2, 7] == dx[0, 7]).all()) and float(dx[0, 9]) > 0
    check_route_grad(dx[-2:].cpu(), tail, got[0][-2:].cpu(), dw[-2:].cpu())


# ---- gradient of the weights ------------------------------------------------------------------------------------------

def grad_ref(x, ids, dw, score, renormalise, scale):
    """(dlogits, an upper bound of its error without the output's rounding) in 64 bits; x [N, K], ids, dw [N, S]."""
    n, K = x.shape
    S = ids.shape[1]
    x, dw = x.double(), dw.double() * float(torch.tensor(scale, dtype=F32))
    live = (ids >= 0) & (ids < K)
    at = torch.where(live, ids.long(), 0)
    dw = torch.where(live, dw, 0.0)
    z = torch.where(live, x.gather(1, at), -math.inf)
    w, R = weights_ref(x, torch.where(live, ids.long(), -1), z, score, renormalise)
    rel = rel_of(R, K, S)
    out, tol = (torch.zeros(n, K, dtype=torch.float64, device=x.device) for _ in range(2))
    if score == "softmax" and not renormalise:
        some = live.any(-1, keepdim=True)
        p = torch.where(some, torch.softmax(torch.where(some, x, 0.0), -1), 0.0)
        top = torch.where(some, x, 0.0).amax(-1, keepdim=True)
        far = torch.where(torch.isfinite(x) & some, (top - x).clamp(max=104), 0.0).amax(-1, keepdim=True)
        rel = rel_of(far, K, S)
        mine = out.scatter_add(1, at, dw)
        size = tol.scatter_add(1, at, dw.abs())
        mean, mag = (p * mine).sum(-1, keepdim=True), (p * size).sum(-1, keepdim=True)
        out = p * (mine - mean)
        tol = p * ((rel + (4 + S) * U) * (size + mag) + (rel + (K / 64 + 40) * U) * mag)
        return out, tol
    if renormalise:
        mean, mag = (w * dw).sum(-1, keepdim=True), (w * dw.abs()).sum(-1, keepdim=True)
        d = w * (dw - mean)
        e = w * ((rel + 4 * U) * (dw.abs() + mag) + (rel + S * U) * mag)
    else:
        d = w * dw
        e = d.abs() * (rel + 4 * U)
    if score == "sigmoid":
        other = torch.where(live, 1.0 / (1.0 + torch.exp(z)), 0.0)
        d, e = d * other, e * other + (d * other).abs() * rel
    m = torch.where(live, d, 0.0), torch.where(live, e, 0.0)
    out.scatter_add_(1, at, m[0])
    tol.scatter_add_(1, at, m[1] + S * U * m[0].abs())
    return out, tol


def check_route_grad(got, x, ids, dw, score="softmax", renormalise=True, scale=1.0, old=None):
    want, tol = grad_ref(x, ids, dw, score, renormalise, scale)
    if old is not None:
        want = want + old.double()
        tol = tol + 2 * U * (old.double().abs() + want.abs())
    live = torch.where((ids >= 0) & (ids < x.shape[1]), dw.abs().double(), 0.0).amax(-1, keepdim=True)
    tol = tol * 1.01 + half_step(got.dtype) * (want.abs() + tol) + tiny(got.dtype) + 2.0 ** -125 * scale * live
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0], float(((got.double() - want).abs() / tol).max()))


def check_all_grads(km, x, ids, z, seed, scales=(1.0,)):
    """Every mode of route_grad for logits x and selections ids (on the CPU), fresh and accumulated."""
    n, K = x.shape
    S = ids.shape[1]
    dw = torch.randn(n, S, generator=gen(seed))
    dw[ids < 0] = math.nan                       # never read into a result
    safe = torch.nan_to_num(dw)
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            for scale in scales:
                kw = dict(score=score, renormalise=renormalise, scale=scale)
                args = cuda(x, ids, z, dw)
                got = km.route_grad(*args, **kw)
                assert got.dtype == x.dtype and got.shape == x.shape
                check_route_grad(got.cpu(), x, ids, safe, **kw)
                old = torch.randn(n, K, generator=gen(seed + 1)).to(x.dtype)
                out = old.cuda()
                assert km.route_grad(*args, out=out, accumulate=True, **kw) is out
                check_route_grad(out.cpu(), x, ids, safe, old=old, **kw)
                live = (ids >= 0) & (ids < K)
                reached = torch.zeros(n, K + 1, dtype=torch.bool).scatter_(1, torch.where(live, ids.long(), K), True)[:, :K]
                if score == "softmax" and not renormalise:
                    reached = reached.any(-1, keepdim=True).expand(n, K)
                assert torch.equal(out.cpu()[~reached], old[~reached])
                fresh = got.cpu()[~reached]
                assert not fresh.any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, K, S", ROUTE_SHAPES)
def test_route_grad(km, dtype, n, K, S):
    x = some_logits(n, K, dtype, n * K)
    valid = torch.rand(n, generator=gen(n)) < 0.9
    ids, _, z = (t.cpu() for t in km.route(x.cuda(), S, valid=valid.cuda()))
    check_all_grads(km, x, ids, z, n, scales=(1.0, 2.5))


@pytest.mark.parametrize("dtype", TYPES)
def test_route_grad_of_rows_with_little_left(km, dtype):
    x = some_logits(50, 12, dtype, 4)
    x[torch.rand(50, 12, generator=gen(3)) < 0.6] = -math.inf
    x[0] = -math.inf
    x[1, 1:] = -math.inf
    ids, _, z = (t.cpu() for t in km.route(x.cuda(), 5))
    assert int((ids == -1).sum()) > 20
    check_all_grads(km, x, ids, z, 1)
    nan = x.clone()
    nan[2] = math.nan
    got = km.route_grad(*cuda(nan, ids, z, torch.ones(50, 5)), renormalise=True).cpu()
    assert torch.isfinite(got).all()             # (logits are not read)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [6, 70, 3000])
def test_route_grad_of_any_ids(km, dtype, K):
    # the same id twice and more, ids outside the choices
    g = gen(K)
    x = some_logits(40, K, dtype, 2, spread=1.0)
    ids = torch.randint(0, min(K, 5), (40, 6), generator=g).to(torch.int32)
    ids[0], ids[1, 0], ids[2] = 3, K, -1
    ids[3] = torch.tensor([K + 7, -(1 << 31), (1 << 31) - 1, -2, K, -1], dtype=torch.int32)
    live = (ids >= 0) & (ids < K)
    z = torch.where(live, x.float().gather(1, torch.where(live, ids.long(), 0)), math.nan)
    n, S = 40, 6
    dw = torch.randn(n, S, generator=g)
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            kw = dict(score=score, renormalise=renormalise)
            got = km.route_grad(*cuda(x, ids, z, dw), **kw).cpu()
            check_route_grad(got, x, ids, dw, **kw)
            old = torch.randn(n, K, generator=g).to(dtype)
            out = km.route_grad(*cuda(x, ids, z, dw), out=old.cuda(), accumulate=True, **kw).cpu()
            check_route_grad(out, x, ids, dw, old=old, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [8, 300, 2100])
def test_route_grad_of_extreme_logits(km, dtype, K):
    fi = torch.finfo(dtype)
    x = some_logits(10, K, dtype, K)
    x[0] = fi.min
    x[1, 1:] = fi.min
    x[2, K - 1] = fi.max
    x[3] = fi.max
    x[4] = -80.0
    x[5] = 60.0
    x[6, 0] = 30.0
    ids, _, z = (t.cpu() for t in km.route(x.cuda(), 3))
    check_all_grads(km, x, ids, z, 5)


def test_route_grad_is_the_weights_derivative(km):
    # central differences of the definition in 64 bits (the ids do not move with the logits)
    x = some_logits(5, 7, F32, 3, spread=1.0)
    dw = torch.randn(5, 3, generator=gen(1))
    h = 1e-5
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            ids, _, z = (t.cpu() for t in km.route(x.cuda(), 3, score=score, renormalise=renormalise))
            want = torch.zeros(5, 7, dtype=torch.float64)
            for k in range(7):
                y = [x.double(), x.double()]
                vals = []
                for s in (1, -1):
                    t = x.double().clone()
                    t[:, k] += s * h
                    w, _ = weights_ref(t, ids.long(), t.gather(1, ids.long()), score, renormalise)
                    vals.append((w * dw.double()).sum(-1) * 1.5)
                want[:, k] = (vals[0] - vals[1]) / (2 * h)
            got = km.route_grad(*cuda(x, ids, z, dw), score=score, renormalise=renormalise, scale=1.5).cpu().double()
            # differences: h^2 times a third derivative below 10, and 64-bit rounding over h; the kernel: fp32
            assert bool(((got - want).abs() <= 1e-9 + 1e-10 + 150 * U * want.abs().max()).all())


@pytest.mark.parametrize("off", [1, 2, 3])
def test_route_grad_at_odd_addresses(km, off):
    for dt in TYPES:
        for n, K in ((77, 5), (77, 16), (50, 200), (3, 9001)):
            x = some_logits(n, K, dt, off)
            buf = torch.zeros(off + n * K, dtype=dt, device="cuda")
            xs = buf[off:].view(n, K)
            xs.copy_(x)
            ids, _, z = km.route(xs, 4)
            dw = torch.randn(n, 4, generator=gen(2))
            for kw in (dict(), dict(renormalise=False)):
                raw = torch.full((off + n * K + 11,), 3.0, dtype=dt, device="cuda")
                out = raw[off:off + n * K].view(n, K)
                km.route_grad(xs, ids, z, dw.cuda(), out=out, **kw)
                check_route_grad(out.cpu(), x, ids.cpu(), dw, **kw)
                assert bool((raw[:off] == 3).all()) and bool((raw[off + n * K:] == 3).all())


# ---- AdamW ----------------------------------------------------------------------------------------------------------------

RATES = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
BLOCK = 256


def f32(x):
    return float(torch.tensor(x, dtype=F32))


def adamw_ref(p, g, m, v, step, lr, betas, eps, weight_decay, decay=1.0, grad_scale=1.0):
    """(p, m, v) and bounds of their errors, in 64 bits, on the CPU."""
    b1, c1, b2, c2 = (f32(t) for t in (betas[0], 1 - betas[0], betas[1], 1 - betas[1]))
    p, g, m, v = (t.double() for t in (p, g, m, v))
    g = g * f32(grad_scale)
    size = b1 * m.abs() + c1 * g.abs()
    m, v = b1 * m + c1 * g, b2 * v + c2 * g * g
    tm, tv = 4 * U * size + 2.0 ** -125, 6 * U * v + 2.0 ** -125
    root = 1 / math.sqrt(1 - betas[1] ** step)
    rate = lr / (1 - betas[0] ** step)
    d = torch.sqrt(v) * root + eps
    q = torch.where(d > 0, m / d, 0.0)
    new = p * (1 - lr * weight_decay * decay) - rate * q
    # of the root: half of v's relative error (a v below the normal range may be gone: its root is then below 2^-62)
    dq = torch.where(d > 0, (16 * U * size + 2.0 ** -125) / d, 0.0) + torch.where(v < 2.0 ** -120, q.abs() * 2.0 ** -60 / d.clamp(
        min=1e-300), 0.0)
    tp = 4 * U * p.abs() + rate * dq + 2 * U * rate * q.abs() + U * new.abs() + 2.0 ** -125
    return (new, m, v), (tp * 1.01, tm * 1.01, tv * 1.01)


def near(got, want, tol, what):
    got, want = got.detach().cpu().double(), want
    both = torch.isnan(got) & torch.isnan(want) | (got == want)
    bad = ~(both | ((got - want).abs() <= tol))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0], float(torch.nan_to_num((got - want).abs() / tol).max()))


def decoded(code, scale):
    n = code.numel()
    x = code.cpu().float().view(-1).double()
    return x * scale.cpu().double().repeat_interleave(BLOCK)[:n]


def check_8bit(code, scale, want, tol, top, half, least, what):
    """Codes and scales of one tensor against the values that they round."""
    n = want.numel()
    pad = -n % BLOCK
    w = torch.nn.functional.pad(want.view(-1), (0, pad)).view(-1, BLOCK)
    t = torch.nn.functional.pad(tol.view(-1), (0, pad)).view(-1, BLOCK)
    fin = torch.where(torch.isfinite(w), w.abs(), 0.0)
    high, thigh = fin.amax(-1, keepdim=True), t.amax(-1, keepdim=True)
    near(scale, (high / top)[:, 0], ((thigh + 2 * U * high) / top)[:, 0] + 2.0 ** -110, f"{what} scale")
    f = high / top
    # half a step of the format (relative, or of its subnormal steps), the type's least positive value, the value's own error
    step = torch.maximum(w.abs() * half, f * least)
    bound = step * (1 + 8 * U) + t + 4 * U * w.abs() + thigh * w.abs() / high.clamp(min=1e-300) + 2.0 ** -99
    near(decoded(code, scale), w.view(-1)[:n], bound.view(-1)[:n], what)


def run_adamw(km, each, pdt, gdt, bits, masters, steps=3, seed=0, offset=0, first=1, spread=1e-2):
    """Steps over tensors of the sizes ``each`` (in buffers `offset` elements past an aligned address), checked one by one
    from the state before."""
    g = gen(seed)
    made = lambda n, dt: torch.zeros(n + offset, dtype=dt, device="cuda")[offset:]  # noqa: E731
    put = lambda t, dt: made(t.numel(), dt).copy_(t)  # noqa: E731
    rand = lambda n: torch.randn(n, generator=g)  # noqa: E731
    W = [put(rand(n), F32) for n in each] if masters else None
    P = [put((W[i].cpu() if masters else rand(n)), pdt) for i, n in enumerate(each)]
    G = [put(rand(n) * spread, gdt) for n in each]
    M, V, scales = km.adamw_states(P, bits)
    if offset:
        M, V = [made(n, torch.uint8 if bits == 8 else F32) for n in each], [made(n, torch.uint8 if bits == 8 else F32) for n in each]
        if bits == 8:
            M, V = [t.view(torch.float8_e4m3fn) for t in M], [t.view(torch.float8_e5m2) for t in V]
    decay = [0.5 * (i % 3) for i in range(len(each))]
    plan = km.adamw_plan(P, G, M, V, scales=scales, masters=W, decay=decay)
    for k in range(first, first + steps):
        for t in G:
            t.copy_(rand(t.numel()) * spread * torch.exp(rand(t.numel()) * 2))
        old = [[t.cpu().clone() for t in ts] for ts in ((W or P), G)]
        m0 = [decoded(M[i], scales[0][i]) if bits == 8 else M[i].cpu().clone() for i in range(len(each))]
        v0 = [decoded(V[i], scales[1][i]) if bits == 8 else V[i].cpu().clone() for i in range(len(each))]
        km.adamw(plan, step=k, **RATES)
        for i, n in enumerate(each):
            (p, m, v), (tp, tm, tv) = adamw_ref(old[0][i], old[1][i], m0[i], v0[i], k, decay=decay[i], **RATES)
            if bits == 8:  # what was decoded has a rounding of its own
                tm, tv = tm + 2 * U * m0[i].abs(), tv + 2 * U * v0[i].abs()
                tp = tp + RATES["lr"] / (1 - 0.9 ** k) * 8 * U * (p.abs() + 10)
                check_8bit(M[i], scales[0][i], m, tm, 256.0, 2.0 ** -4, 2.0 ** -10, "m")
                check_8bit(V[i], scales[1][i], v, tv, 32768.0, 2.0 ** -3, 2.0 ** -16, "v")
                pos = v > 2.0 ** -98
                assert bool((decoded(V[i], scales[1][i])[pos] > 0).all())
            else:
                near(M[i], m, tm, "m")
                near(V[i], v, tv, "v")
            if masters:
                near(W[i], p, tp, "master")
                assert torch.equal(P[i].cpu(), W[i].cpu().to(pdt))
            else:
                near(P[i], p, tp + half_step(pdt) * (p.abs() + tp) * (pdt != F32) + tiny(pdt), "p")
    return P, M, V


SIZES = [[1], [255, 256, 257], [4096], [4095, 1, 4097, 0, 12288, 3], [70001]]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt, gdt, masters", [(F32, F32, False), (F32, BF16, False), (F32, F16, False), (BF16, BF16, True),
                                               (BF16, F32, True), (BF16, BF16, False), (F16, F16, True), (F16, F32, False),
                                               (F16, BF16, False), (BF16, F16, True)])
@pytest.mark.parametrize("each", SIZES)
def test_adamw(km, each, pdt, gdt, masters, bits):
    run_adamw(km, each, pdt, gdt, bits, masters, seed=len(each))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_adamw_at_odd_addresses(km, offset, bits):
    run_adamw(km, [4096, 300, 8191], BF16, F16, bits, True, offset=offset)
    run_adamw(km, [4096, 300], F32, F32, bits, False, offset=offset)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_far_steps_and_sizes(km, bits):
    run_adamw(km, [5000], F32, F32, bits, False, first=100000, steps=2)
    run_adamw(km, [5000], F32, F32, bits, False, spread=1e-9)
    run_adamw(km, [5000], F32, F32, bits, False, spread=1e3)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_over_many_tensors_of_mixed_types(km, bits):
    g = gen(5)
    each = [int(n) for n in torch.randint(1, 3000, (300,), generator=g)]
    kinds = [(TYPES[i % 3], TYPES[(i // 3) % 3], i % 3 != 0 and i % 2 == 0) for i in range(300)]
    P = [torch.randn(n, generator=g).to(a).cuda() for n, (a, _, _) in zip(each, kinds)]
    G = [torch.randn(n, generator=g).to(b).cuda() for n, (_, b, _) in zip(each, kinds)]
    W = [p.float() if w else None for p, (_, _, w) in zip(P, kinds)]
    M, V, scales = km.adamw_states(P, bits)
    want = [adamw_ref((w if w is not None else p).cpu(), gr.cpu(), torch.zeros(n), torch.zeros(n), 1, **RATES)
            for p, gr, w, n in zip(P, G, W, each)]
    km.adamw(km.adamw_plan(P, G, M, V, scales=scales, masters=W), step=1, **RATES)
    for i, ((p, m, v), (tp, tm, tv)) in enumerate(want):
        near(P[i], p, 2 * tp + half_step(kinds[i][0]) * (p.abs() + tp) + tiny(kinds[i][0]), i)
        if bits == 32:
            near(M[i], m, tm, i)
            near(V[i], v, tv, i)
        else:
            check_8bit(M[i], scales[0][i], m, tm, 256.0, 2.0 ** -4, 2.0 ** -10, i)
            check_8bit(V[i], scales[1][i], v, tv, 32768.0, 2.0 ** -3, 2.0 ** -16, i)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_nan_and_infinities(km, bits):
    n = 1000
    p, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda") * 0.5
    g[7], g[300], g[301] = math.nan, math.inf, -math.inf
    M, V, scales = km.adamw_states([p], bits)
    plan = km.adamw_plan([p], [g], M, V, scales=scales)
    km.adamw(plan, step=1, **RATES)
    bad = torch.zeros(n, dtype=torch.bool)
    bad[[7, 300, 301]] = True
    for t in (p, M[0].float(), V[0].float(), *([s[0] for s in scales] if scales else [])):
        if t.numel() == n:
            ok = torch.isfinite(t.cpu())
            assert bool(ok[~bad].all()) and not ok[7] and not (t is not p and ok[300])
            assert bool((t.cpu()[~bad] == t.cpu()[0]).all())
        else:
            assert bool(torch.isfinite(t).all())
    # nothing has moved: no step, and with eps 0 no NaN
    q, z = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    M, V, scales = km.adamw_states([q], bits)
    km.adamw(km.adamw_plan([q], [z], M, V, scales=scales), lr=0.1, step=1, eps=0.0, weight_decay=0.0)
    assert bool((q == 1).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_scalars_on_the_device(km, bits):
    def fresh():
        p = torch.linspace(-1, 1, 9000).cuda()
        g = torch.linspace(3, -2, 9000).cuda()
        M, V, s = km.adamw_states([p], bits)
        return p, M[0], V[0], km.adamw_plan([p], [g], M, V, scales=s)
    a, b = fresh(), fresh()
    lr, step = torch.tensor([f32(1e-2)], device="cuda"), torch.tensor(1, device="cuda")
    gs, skip = torch.tensor([0.25], device="cuda"), torch.tensor([False], device="cuda")
    for k in range(1, 4):
        km.adamw(a[3], step=k, grad_scale=gs, **{**RATES, "lr": f32(1e-2)})
        km.adamw(b[3], step=step, grad_scale=gs, skip=skip, **{**RATES, "lr": lr})
        step += 1
        # (the host's pow and the device's may differ in the last bit of 64, which the rounding to 32 may show)
        assert bool(((a[0] - b[0]).abs() <= 4 * U * (a[0].abs() + 0.02)).all())
    kept = [t.clone() for t in b[:3]]
    skip.fill_(True)
    km.adamw(b[3], step=step, skip=skip, lr=lr)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(kept, b[:3]))


def test_adamw_offsets_past_32_bits(km):
    n = (1 << 31) + 4099
    p = torch.zeros(n, dtype=BF16, device="cuda")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-5:] = 1.0
    g[:3] = -1.0
    M, V, scales = km.adamw_states([p], 8)
    km.adamw(km.adamw_plan([p], [g], M, V, scales=scales), lr=0.5, step=1, weight_decay=0.0)
    assert bool((p[-5:] == -0.5).all()) and bool((p[:3] == 0.5).all()) and not p[3:-5].any()
    assert float(decoded(M[0][-3:], scales[0][0][-1:])[0]) == pytest.approx(0.1, rel=1e-6)


# ---- how they are called ------------------------------------------------------------------------------------------------

def test_refusals_on_the_gpu(km):
    x = torch.zeros(6, 8, device="cuda")
    i, f = torch.zeros(6, 2, dtype=torch.int32, device="cuda"), torch.zeros(6, 2, device="cuda")
    M, V, _ = km.adamw_states([x])
    E = km.KMeansError
    for call in (lambda: km.route(x, 0), lambda: km.route(x, 9), lambda: km.route(x, 65), lambda: km.route(x.double(), 2),
                 lambda: km.route(x[:, ::2], 2), lambda: km.route(x[0], 2), lambda: km.route(x, 2, score="tanh"),
                 lambda: km.route(x, 2, score=0), lambda: km.route(x, 2, bias=torch.zeros(7, device="cuda")),
                 lambda: km.route(x, 2, bias=torch.zeros(8)), lambda: km.route(x, 2, groups=3),
                 lambda: km.route(x, 2, groups=4, top_groups=5), lambda: km.route(x, 2, group_best=3),
                 lambda: km.route(x, 2, valid=torch.zeros(6, device="cuda")),
                 lambda: km.route_grad(x, i.long(), f, f), lambda: km.route_grad(x, i[:3], f, f),
                 lambda: km.route_grad(x, i, f[:, :1].contiguous(), f), lambda: km.route_grad(x, i, f, f, accumulate=True),
                 lambda: km.route_grad(x, i, f, f, out=x.half()), lambda: km.route_grad(x, i, f, f.double()),
                 lambda: km.route_grad(x, i, f, f, out=x, renormalise=False),
                 lambda: km.adamw_plan([x], [x], [x], V), lambda: km.adamw_plan([x], [x.t()], M, V),
                 lambda: km.adamw_plan([x], [x.double()], M, V), lambda: km.adamw_plan([x.half()], [x], [x.half()], V),
                 lambda: km.adamw_plan([x, x], [x, x], M * 2, V * 2), lambda: km.adamw_plan([x], [x], M, M),
                 lambda: km.adamw_plan([x], [f], M, V), lambda: km.adamw_plan([x], [f], M, V, masters=[f]),
                 lambda: km.adamw_plan([x], [x.clone()], M, V, masters=[x.clone()]),
                 lambda: km.adamw_plan([x], [x.clone()], M, V, scales=([f], [f]))):
        with pytest.raises(E):
            call()
    # overlaps across launches of different types
    h = torch.zeros(6, 8, device="cuda", dtype=F16)
    M2, V2, _ = km.adamw_states([x, h])
    with pytest.raises(E, match="overlaps"):
        km.adamw_plan([x, h], [x.clone(), h.clone()], [M2[0], M2[0]], V2)
    plan = km.adamw_plan([x], [x.clone()], M, V)
    one = torch.ones(1, device="cuda")
    for kw in (dict(lr=0.1, step=0), dict(lr=math.inf, step=1), dict(lr=one.double(), step=1), dict(lr=one, step=one),
               dict(lr=0.1, step=1, grad_scale=2.0), dict(lr=0.1, step=1, grad_scale=one.repeat(2)),
               dict(lr=0.1, step=1, skip=True), dict(lr=0.1, step=1, skip=one), dict(lr=0.1, step=1, betas=(1.0, 0.9)),
               dict(lr=0.1, step=1, eps=-1.0), dict(lr=one.cpu(), step=1)):
        with pytest.raises(E):
            km.adamw(plan, **kw)
    assert not x.any()


def test_no_rows(km):
    x = torch.zeros(0, 8, device="cuda")
    ids, w, z = km.route(x, 3)
    assert ids.shape == w.shape == z.shape == (0, 3)
    assert km.route_grad(x, ids, z, w).shape == (0, 8)
    e = torch.zeros(0, device="cuda")
    M, V, _ = km.adamw_states([e, x])
    km.adamw(km.adamw_plan([e, x], [e, x], M, V), lr=0.1, step=1)


def test_batched_rows_are_rows(km):
    x = some_logits(30, 24, BF16, 1)
    valid = torch.rand(30, generator=gen(2)) < 0.7
    flat = km.route(x.cuda(), 4, valid=valid.cuda(), score="sigmoid")
    both = km.route(x.cuda().view(3, 10, 24), 4, valid=valid.cuda().view(3, 10), score="sigmoid")
    assert both[0].shape == (3, 10, 4)
    assert all(torch.equal(a.view(30, 4), b) for a, b in zip(both, flat))
    dw = torch.randn(30, 4, generator=gen(3)).cuda()
    a = km.route_grad(x.cuda(), flat[0], flat[2], dw, score="sigmoid")
    b = km.route_grad(x.cuda().view(3, 10, 24), both[0], both[2], dw.view(3, 10, 4), score="sigmoid")
    assert b.shape == (3, 10, 24) and torch.equal(a, b.view(30, 24))


def a_state(km, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = {"x": r(700, 48).to(F16), "bias": (r(48) * 10).round() * 0.001, "dw": r(700, 4),
         "valid": torch.rand(700, generator=g, device="cuda") < 0.9, "old": r(700, 48).to(F16),
         "p": r(9000).to(BF16), "w": None, "q": r(77), "gp": r(9000).to(BF16), "gq": r(77)}
    s["w"] = s["p"].float()
    return s


def operators(km, s, plans=None, stream=None):
    """Each operator once on copies of what the state holds; all their outputs."""
    ids, w, z = km.route(s["x"], 4, score="sigmoid", bias=s["bias"], groups=6, top_groups=3, valid=s["valid"], stream=stream)
    other = km.route(s["x"], 4, renormalise=False, stream=stream)
    dx = km.route_grad(s["x"], ids, z, s["dw"], score="sigmoid", stream=stream)
    dy = km.route_grad(s["x"], other[0], other[2], s["dw"], renormalise=False, stream=stream)
    acc = s["old"].clone() if stream is None else s["acc"]
    km.route_grad(s["x"], ids, z, s["dw"], score="sigmoid", out=acc, accumulate=True, stream=stream)
    return [ids, w, z, *other, dx, dy, acc]


def stepped(km, s, bits, stream=None, steps=2):
    p, w, q = s["p"].clone(), s["w"].clone(), s["q"].clone()
    M, V, scales = km.adamw_states([p, q], bits)
    plan = km.adamw_plan([p, q], [s["gp"], s["gq"]], M, V, scales=scales, masters=[w, None])
    for k in range(1, steps + 1):
        km.adamw(plan, step=k, stream=stream, **RATES)
    return [t.view(torch.uint8) for t in (p, w, q, *M, *V)]


def test_another_stream(km):
    s = a_state(km, 1)
    want = operators(km, s) + stepped(km, s, 8)
    side = torch.cuda.Stream()
    s["acc"] = s["old"].clone()
    side.wait_stream(torch.cuda.current_stream())
    got = operators(km, s, stream=side)
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        got = operators(km, s) + stepped(km, s, 8)
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    # a plan made on one stream and used on another
    p, g = torch.ones(5000, device="cuda"), torch.ones(5000, device="cuda")
    M, V, _ = km.adamw_states([p])
    plan = km.adamw_plan([p], [g], M, V)
    torch.cuda.synchronize()
    km.adamw(plan, lr=0.5, step=1, weight_decay=0.0, stream=side)
    side.synchronize()
    assert bool(((p - 0.5).abs() < 1e-6).all())


def test_two_streams_at_once(km):
    states = [a_state(km, 1), a_state(km, 2)]
    want = [[t.clone() for t in operators(km, s) + stepped(km, s, 32)] for s in states]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(operators(km, states[k]) + stepped(km, states[k], 32))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(run, want[k]))


def test_the_same_every_time(km):
    s = a_state(km, 3)
    a = operators(km, s) + stepped(km, s, 8)
    for _ in range(3):
        b = operators(km, s) + stepped(km, s, 8)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_and_replayed(km, bits):
    """A training step with device-side step count and rate, captured once, replayed on new inputs with the program's own
    work between the replays, against the eager steps."""
    states = [a_state(km, k) for k in (1, 2, 3, 4)]
    want = [[t.clone() for t in operators(km, s)] for s in states]
    held = a_state(km, 1)

    def training(s):
        p, w, q = s["p"].clone(), s["w"].clone(), s["q"].clone()
        M, V, scales = km.adamw_states([p, q], bits)
        gp, gq = s["gp"].clone(), s["gq"].clone()
        plan = km.adamw_plan([p, q], [gp, gq], M, V, scales=scales, masters=[w, None])
        return plan, gp, gq, [p, w, q, *M, *V]

    a, b = training(held), training(held)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.tensor([0.01], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        operators(km, held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        got = operators(km, held)
        km.adamw(a[0], **{**RATES, "lr": lr}, step=step)
    for k, turn in enumerate((1, 2, 0, 3)):
        for name, t in states[turn].items():
            held[name].copy_(t)
        for run in (a, b):
            run[1].copy_(states[turn]["gp"])
            run[2].copy_(states[turn]["gq"])
        lr.fill_(0.01 / (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(got, want[turn])), turn
        at = torch.tensor([k + 1], device="cuda")
        km.adamw(b[0], **{**RATES, "lr": torch.tensor([0.01], device="cuda") / (k + 1)}, step=at)
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[3], b[3])), turn
        eager = operators(km, states[2])
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(eager, want[2]))


def test_a_routers_and_codebooks_training_step(km):
    """Route, look up, balance, differentiate and step, as a codebook with a learned router is trained, against the same
    step by torch's own differentiation in 64 bits on the CPU with the ids held fixed."""
    g = gen(11)
    N, K, D, S, H = 600, 48, 40, 3, 24
    X = torch.randn(N, H, generator=g)
    W = torch.randn(H, K, generator=g) * 0.3
    C = torch.randn(K, D, generator=g)
    Y = torch.randn(N, D, generator=g)
    bias = some_bias(K, 1)
    valid = torch.rand(N, generator=g) < 0.9
    alpha = 0.02
    Xg, Wg, Cg, Yg, bg, vg = cuda(X, W, C, Y, bias, valid)
    live = vg[:, None].float()
    logits = Xg @ Wg
    ids, w, z = km.route(logits, S, bias=bg, valid=vg, scale=1.5)
    rows = km.embed(Cg, ids.view(-1)).view(N, S, D)
    out = (w[..., None] * rows).sum(1)
    dout = (out - Yg) * live * (2.0 / N)
    dweights = (dout[:, None, :] * rows).sum(-1)
    loss, counts, prob, saved = km.balance(logits, ids, valid=vg)
    dlogits = km.balance_grad(logits, saved, torch.full((1,), alpha, device="cuda"))
    km.route_grad(logits, ids, z, dweights.contiguous(), scale=1.5, out=dlogits, accumulate=True)
    dC = km.embed_grad((w[..., None] * dout[:, None, :]).reshape(N * S, D).contiguous(), ids.view(-1), K)
    dW = Xg.t().contiguous() @ dlogits
    # in 64 bits
    Wd, Cd = W.double().requires_grad_(), C.double().requires_grad_()
    x = X.double() @ Wd
    at = ids.cpu().long()
    assert bool((at[valid] >= 0).all()) and bool((at[~valid] == -1).all())
    assert int(counts.sum()) == S * int(valid.sum())
    p = torch.softmax(x, -1)
    share = torch.where(valid[:, None], p.gather(1, at.clamp(min=0)), 0.0)
    weights = 1.5 * share / share.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (weights[..., None] * Cd[at.clamp(min=0)]).sum(1)
    T = int(valid.sum())
    bal = K * (counts.cpu().double() / (S * T) * p[valid].sum(0) / T).sum()
    total = ((o - Y.double())[valid].square().sum()) / N + alpha * bal
    total.backward()
    # fp32 products over H, N and D terms, exponentials of logits below 10: a few hundred roundings of the magnitudes
    for got, want in ((dW, Wd.grad), (dC, Cd.grad)):
        assert float((got.cpu().double() - want).abs().max()) <= 600 * U * float(want.abs().max() + want.abs().mean() * 10)
    M, V, _ = km.adamw_states([Wg, Cg])
    plan = km.adamw_plan([Wg, Cg], [dW, dC], M, V)
    want = [adamw_ref(p0, d.cpu(), torch.zeros_like(p0), torch.zeros_like(p0), 1, **RATES) for p0, d in ((W, dW), (C, dC))]
    km.adamw(plan, step=1, **RATES)
    for t, ((p1, _, _), (tol, _, _)) in zip((Wg, Cg), want):
        near(t, p1, tol, "stepped")
