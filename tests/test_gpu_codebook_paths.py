"""The codebook operators on the paths that tests/test_gpu_codebook.py does not reach (definitions and tolerances there;
u = 2^-24)."""

import math

import pytest
import torch

from tests.test_gpu_codebook import BF16, F16, F32, TYPES, U, half_step, km, tiny  # noqa: F401  (km is the fixture)

pytestmark = pytest.mark.gpu


def pieces(n, size=1 << 28):
    for at in range(0, n, size):
        yield at, min(n, at + size)


def test_balance_at_the_largest_k(km):  # noqa: F811
    # Column counts next to 2^31.  With logits of 0 (and, for the gradient, which takes nothing but the live rows from
    # it, an lse of 0) a thread adds fewer than 2^24 ones, exactly; 8 levels of joins then round both sums.
    K = (1 << 31) - 8
    x = torch.zeros(1, K, dtype=BF16, device="cuda")
    out = [0, 7, 1 << 30, K - 2049, K - 3]
    named = [5, K - 1]
    x[0, out] = -math.inf
    left = K - len(out)
    loss, counts, prob, (lse, coef) = km.balance(x, torch.tensor([named], dtype=torch.int32, device="cuda"))
    assert int(counts.sum(dtype=torch.int64)) == 2 and counts[named].tolist() == [1, 1]
    assert abs(float(lse[0]) - math.log(left)) <= 20 * U * math.log(left)
    assert abs(float(loss) - K / left) <= 16 * U * K / left
    assert not prob[out].any()
    # K / 2 has 28 bits, the fp32 coef 24: one rounding
    assert all(abs(c - K / 2) <= U * K / 2 for c in coef[named].tolist()) and int((coef != 0).sum()) == 2
    near = sum(int(((prob[a:b].double() * left - 1).abs() <= 16 * U).sum()) for a, b in pieces(K))
    assert near == left
    del prob, counts
    dl = 1024.0
    dx = km.balance_grad(x, (torch.zeros_like(lse), coef), torch.full((1,), dl, device="cuda"))[0]
    assert not dx[out].any()
    mean = K / left                                      # of coef under p
    tol = 64 * U + half_step(BF16) * (1 + 64 * U)
    want = dl / left * (K / 2 - mean)
    assert all(abs(float(v) - want) <= tol * want for v in dx[named])
    want = dl / left * mean
    near = sum(int(((dx[a:b].float() + want).abs() <= tol * want).sum()) for a, b in pieces(K))
    assert near == left - 2
    del dx, coef, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype, K", [(BF16, 1 << 24), (F16, (1 << 22) + 5), (F32, (1 << 23) + 4)])
def test_balance_sums_of_very_long_rows(km, dtype, K):  # noqa: F811
    # rows of equal logits but for one and for the first 2,048 (below a thread's own maximum every addition of a long
    # sum rounds the same way), and a random row
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    x = torch.full((3, K), -2.0, dtype=dtype, device="cuda")
    x[0, 3] = 0
    x[2, :2048] = 0
    x[1] = torch.randn(K, generator=g, device="cuda") * 2
    labels = torch.randint(0, K, (3, 3), generator=g, device="cuda", dtype=torch.int32)
    dl = torch.full((1,), float(K), device="cuda")
    loss, counts, prob, (lse, coef) = km.balance(x, labels)
    dx = km.balance_grad(x, (lse, coef), dl)
    z = x.double()
    p = torch.softmax(z, -1)
    R = z.amax(-1, keepdim=True) - z.amin(-1, keepdim=True)
    # an exponential (R + 4) u; a thread's sum of up to 256 fp32 values before 64 bits take it over, then 10 roundings
    row = (R + 4 + 256 + 10) * U
    want = torch.logsumexp(z, -1)
    assert bool(((lse.double() - want).abs() <= row[:, 0] + 3 * U * want.abs()).all())
    rel = (row + (R + 8) * U).max()
    want = p.mean(0)
    assert bool(((prob.double() - want).abs() <= rel * want).all())
    want = K / 3 * (counts.double() / 3 * want).sum()
    assert float((loss.double() - want).abs()) <= float((rel + U) * want)
    c = coef.double()
    dot = (p * c).sum(-1, keepdim=True)
    want = float(dl) * p * (c - dot)
    tol = float(dl) * p * ((rel + 4 * U) * (c + dot) + rel * dot + 266 * U * dot)
    tol = tol * 1.01 + half_step(dtype) * (want.abs() + tol) + tiny(dtype) + 2.0 ** -126 * float(dl) * (c + dot)
    # (a labelled column's gradient may be past the type's range)
    over = torch.isinf(dx) & (want.abs() + tol >= torch.finfo(dtype).max)
    assert bool((((dx.double() - want).abs() <= tol) | over).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [3, 64, 189, 1500, 9000, 16500, 20001])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_balance_rows_without_a_softmax(km, dtype, K, bad):  # noqa: F811
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    x = torch.randn(2, 9, K, generator=g, device="cuda").to(dtype)
    labels = torch.randint(0, K, (2, 9), generator=g, device="cuda", dtype=torch.int32)
    valid = torch.ones(2, 9, dtype=torch.bool, device="cuda")
    valid[0, 2] = False
    x[0, 2, K // 2] = bad                                # of an invalid row: no consequence
    plain = x.clone()
    x[1, 4, K - 1] = bad
    want = km.balance(plain, labels, valid=valid)
    got = km.balance(x, labels, valid=valid)
    assert torch.equal(got[1], want[1]) and torch.equal(got[3][1], want[3][1])
    assert torch.equal(got[0][0], want[0][0]) and bool(torch.isnan(got[0][1]))
    assert torch.equal(got[2][0], want[2][0]) and bool(torch.isnan(got[2][1]).all())
    rest = torch.ones(2, 9, dtype=torch.bool, device="cuda")
    rest[1, 4] = False
    assert bool(torch.isnan(got[3][0][1, 4])) and torch.equal(got[3][0][rest], want[3][0][rest])
    assert bool(torch.isinf(got[3][0][0, 2]))
    dl = torch.full((2,), 9.0, device="cuda")
    dx, dw = km.balance_grad(x, got[3], dl), km.balance_grad(plain, want[3], dl)
    assert bool(torch.isnan(dx[1, 4]).all()) and torch.equal(dx[rest], dw[rest]) and not dx[0, 2].any()


# ---- gradient of the lookup ------------------------------------------------------------------------------------------

def ids_on_gpu(n, K, kind, g):
    r = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if kind == "one":
        ids = torch.full((n,), K // 2, device="cuda")
    elif kind == "hot":                                  # half of the rows on a few entries, a tenth on none
        ids = (r ** 6 * K).long()
        ids[torch.rand(n, generator=g, device="cuda") < 0.1] = -1
    elif kind == "runs":                                 # 15 to 17 rows an entry: segments that end at and around a unit's edge
        ids = torch.arange(n, device="cuda") // 16 % K
        ids[::31] = (ids[::31] + 1) % K
        ids = ids[torch.randperm(n, generator=g, device="cuda")]
    else:                                                # ids outside the table among them
        ids = (r * 1.1 * K).long()
        ids[::97] = -(1 << 31)
    return ids.to(torch.int32)


def check_grad_on_gpu(got, dout, ids, K, scale, old=None):
    """got [K, D] against the definition in 64 bits, with the tolerance of test_gpu_codebook.check_grad."""
    D = dout.shape[1]
    hit = ((ids >= 0) & (ids < K)).nonzero()[:, 0]
    key, order = torch.sort(ids[hit].long(), stable=True)
    rows = hit[order]
    ends = torch.searchsorted(key, torch.arange(K + 1, device="cuda"))
    m = ends[1:] - ends[:-1]
    s32 = float(torch.tensor(scale, dtype=F32))
    for a in range(0, D, 256):                           # columns in pieces
        x = dout[:, a:a + 256][rows].double()
        total, mag = (torch.segment_reduce(v, "sum", lengths=m, axis=0, initial=0.0) for v in (x, x.abs()))
        y = got[:, a:a + 256]
        want = s32 * total
        tol = (m + 1).double()[:, None] * U * abs(s32) * mag * 1.01
        bare = m == 0
        if old is None:
            assert not y[bare].any()
        else:
            o = old[:, a:a + 256]
            assert torch.equal(y[bare], o[bare])
            want = want + o.double()
            tol = tol + 2 * U * (want.abs() + abs(s32) * mag)
        tol = tol + half_step(got.dtype) * (want.abs() + tol) + tiny(got.dtype)
        bad = (y.double() - want).abs() > tol
        assert not bool(bad.any()), (a, int(bad.sum()))


def run_grad(km, n, K, D, kind, of, to):
    g = torch.Generator(device="cuda")
    g.manual_seed(n * 7 + D)
    dout = torch.randn(n, D, generator=g, device="cuda").to(of)
    ids = ids_on_gpu(n, K, kind, g)
    got = km.embed_grad(dout, ids, K, scale=0.3, grad_dtype=to)
    check_grad_on_gpu(got, dout, ids, K, 0.3)
    old = torch.randn(K, D, generator=g, device="cuda").to(to)
    buf = old.clone()
    km.embed_grad(dout, ids, K, scale=1.5, out=buf, accumulate=True)
    check_grad_on_gpu(buf, dout, ids, K, 1.5, old)


@pytest.mark.parametrize("of, to", [(BF16, F32), (F16, F16), (F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("n, K, D, kind", [
    # rows of whole vectors wider than a wave: one slab, a second one of a single vector, several; rows of 4 elements at
    # a time and of single ones; joins inside the workgroup and of one and two levels behind it
    (300, 40, 512, "mixed"), (300, 9, 520, "hot"), (2000, 100, 1024, "runs"), (4099, 700, 1024, "hot"),
    (5000, 3, 2048, "mixed"), (6000, 1, 1024, "one"), (9001, 500, 1028, "runs"), (16384, 900, 1024, "runs"),
    (20011, 60000, 520, "hot"), (20011, 1300, 1536, "runs"), (70001, 1000, 1024, "hot"), (70001, 2, 1024, "one"),
    (70001, 90, 1029, "hot")])
def test_embed_grad_of_wide_rows(km, of, to, n, K, D, kind):  # noqa: F811
    run_grad(km, n, K, D, kind, of, to)


@pytest.mark.parametrize("n", [256, 257, 1024, 1025, 2048, 2049, 4096, 4097, 8192, 8193, 16384, 16385])
@pytest.mark.parametrize("K", [600, 200000])
def test_embed_grad_at_its_limits(km, n, K):  # noqa: F811
    run_grad(km, n, K, 1024 if K == 600 else 136, "hot", BF16, F32)


@pytest.mark.parametrize("n", [1 << 23, (1 << 23) + 1, (1 << 23) + 4099])
@pytest.mark.parametrize("K", [5000, 65536, 90000])
def test_embed_grad_of_more_rows_than_a_packed_word_holds(km, n, K):  # noqa: F811
    run_grad(km, n, K, 8, "mixed", BF16, F32)


@pytest.mark.parametrize("of, to", [(BF16, F32), (F32, F32), (F16, F16)])
@pytest.mark.parametrize("D", [1, 16, 40, 100, 264])
def test_embed_grad_of_narrow_rows_at_a_large_n(km, of, to, D):  # noqa: F811
    run_grad(km, 700003, 30000, D, "hot", of, to)


# ---- balance: rings that turn, blocks that fold, chunks that join --------------------------------------------------------

def balance_depths(K, steps):
    """(row, column): roundings of a row's sum and of a column's.  K <= 16,384: a lane adds K / 64 + 16 values at most,
    then 6 levels and up to 16 waves; a column has blocks of 64 rows, then the blocks, 6 levels and one rounding of a
    chunk.  Longer rows: a load's 8 values, fp64, 10 roundings; a column has the 64 rows of a chunk and its rounding."""
    if K > 16384:
        return 20, 66
    return K / 64 + 40, 64 + -(-steps // 64) + 8


def check_balance_on_gpu(km, B, N, K, S, dtype, steps, spread=3.0, masked=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + K)
    x = torch.empty(B, N, K, dtype=dtype, device="cuda")
    flat = x.view(-1, K)
    rows = max(1, (1 << 25) // K)
    for a, b in pieces(B * N, rows):
        flat[a:b] = torch.randn(b - a, K, generator=g, device="cuda") * spread
    labels = torch.randint(-1, K, (B, N, S), generator=g, device="cuda", dtype=torch.int32)
    valid = torch.rand(B, N, generator=g, device="cuda") < 0.85
    one = B == 1
    if masked:
        x[~valid] = math.nan
    else:
        valid[:] = True
    got = km.balance(x[0] if one else x, labels[0] if one else labels, valid=(valid[0] if one else valid) if masked else None)
    loss, counts, prob, (lse, coef) = got
    dl = torch.rand(B, generator=g, device="cuda") + N
    dx = km.balance_grad(x[0] if one else x, (lse, coef), dl).view(-1, K)
    counts, prob, coef, lse = counts.view(B, K), prob.view(B, K), coef.view(B, K), lse.view(-1)
    row, col = balance_depths(K, steps)
    T = valid.sum(1).double()
    named = torch.where(valid[..., None] & (labels >= 0), labels.long() + torch.arange(B, device="cuda")[:, None, None] * K, B * K)
    want = torch.bincount(named.view(-1), minlength=B * K + 1)[:-1].view(B, K)
    assert torch.equal(counts.long(), want)
    share = want.double() * (K / S) / T[:, None]
    assert bool(((coef.double() - share / T[:, None]).abs() <= 2 * U * share / T[:, None]).all())
    total = torch.zeros(B, K, dtype=torch.float64, device="cuda")
    at = torch.arange(B * N, device="cuda") // N
    live = valid.view(-1)
    most = torch.zeros((), dtype=torch.float64, device="cuda")
    c64 = coef.double()
    for a, b in pieces(B * N, rows):
        on = live[a:b]
        z = torch.where(on[:, None], flat[a:b].double(), 0.0)
        R = z.amax(-1, keepdim=True) - z.amin(-1, keepdim=True)
        most = torch.maximum(most, R.max())
        p = torch.softmax(z, -1) * on[:, None]
        r = torch.logsumexp(z, -1)
        assert bool(torch.isposinf(lse[a:b][~on]).all())
        tol = (R[:, 0] + 4 + row) * U + 3 * U * (r.abs() + math.log(K) + 1)
        assert bool(((lse[a:b].double() - r).abs() <= tol)[on].all())
        for q in range(int(at[a]), int(at[b - 1]) + 1):
            total[q] += p[max(0, q * N - a):(q + 1) * N - a].sum(0)
        c = c64[at[a:b]]
        d = dl.double()[at[a:b], None]
        dot = (p * c).sum(-1, keepdim=True)
        want = d * p * (c - dot)
        rel = (2 * R + 8 + row) * U
        tol = d * p * ((rel + 4 * U) * (c + dot) + (rel + row * U) * dot)
        tol = tol * 1.01 + half_step(dtype) * (want.abs() + tol) + tiny(dtype) + 2.0 ** -126 * d * (c + dot)
        out = dx[a:b].double()
        bad = ~((out - want).abs() <= tol)
        assert not bool(bad.any()), (a, int(bad.sum()))
        assert not out[~on].any()
    prob64 = total / T[:, None]
    rel = (2 * most + 8 + row + col) * U
    assert bool(((prob.double() - prob64).abs() <= rel * prob64).all())
    want = (share * prob64).sum(1)
    assert bool(((loss.double() - want).abs() <= (rel + U) * want).all())


# steps: rows a team takes one after another (chosen so that a ring of 4 turns, a block of 64 folds, several chunks join)
@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B, N, K, S, steps", [
    (1, 50003, 1024, 1, 7), (1, 50003, 520, 2, 7), (1, 50003, 1001, 1, 7), (3, 20001, 700, 3, 8), (2, 140001, 250, 2, 18),
    (1, 1000003, 8, 2, 4), (1, 300007, 100, 2, 10), (1, 9001, 2048, 1, 5), (1, 20001, 3999, 2, 10), (1, 9001, 8192, 1, 9),
    (1, 5003, 8200, 2, 10), (1, 4001, 12345, 1, 8), (2100, 23, 200, 2, 4), (2100, 131, 129, 1, 17)])
def test_balance_of_many_steps(km, dtype, B, N, K, S, steps, masked):  # noqa: F811
    check_balance_on_gpu(km, B, N, K, S, dtype, steps, masked=masked)


@pytest.mark.parametrize("B, N, K, S, steps", [(2100, 1201, 100, 1, 76), (2050, 600, 200, 2, 75), (2050, 140, 1000, 1, 35),
                                               (2050, 290, 601, 2, 73), (1, 600011, 1024, 1, 74), (1, 140003, 2048, 1, 69),
                                               (1, 70001, 8192, 1, 69), (1, 36007, 12345, 1, 71)])
def test_balance_of_more_steps_than_a_block(km, B, N, K, S, steps):  # noqa: F811
    check_balance_on_gpu(km, B, N, K, S, BF16, steps)


@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B, N, K, S", [(1, 64, 16385, 1), (1, 65, 16392, 2), (3, 129, 20001, 1), (2, 200, 40000, 3),
                                        (1, 4100, 16389, 1), (1, 1, 1000001, 2), (5, 3, 50257, 1)])
def test_balance_of_long_rows(km, dtype, B, N, K, S, masked):  # noqa: F811
    check_balance_on_gpu(km, B, N, K, S, dtype, 0, masked=masked)
