"""The codebook operators on the GPU against their definitions in 64 bits.

Tolerances count roundings (u = 2^-24, half a step of fp32; half a step of the output's type is eps / 2):
  embed         one fp32 product, then one rounding: bit for bit the same two steps in torch.
  embed_grad    a sum of m values in any order is off by at most (m - 1) u times the sum of their magnitudes; the scale
                and the addition to the old value add u each, the output's type half a step (and, for fp16, half of its
                smallest step 2^-24).
  balance       with R the largest |logit - maximum| that still leaves a probability (exp of less than -104 is 0 in
                fp32), an exponential is off by (R + 4) u relative (the difference's rounding, its scaling, exp itself), a
                row's sum by another (K / 64 + 24) u (lanes add at most K / 64 + 16 values one after another, then 6 levels
                of pairs), a column's by ROWS u more (blocks of 64 rows added one after another), by one u a block (4 at
                most here) and by 6 over a wave's lanes, which the 24 of the row's sum and the 8 leave room for (the row's
                own sums of at most 16 values and 6 levels take 22 of them only where a lane has 16 values, and then a
                wave holds one row).
  balance_grad  p is off by an exponential and a row's sum as above; the mean of coef under p by that and a sum's depth;
                the difference, the products and the output's type add 4 u and half a step.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROWS = 64   # rows that one fp32 column sum may hold before it is added in 64 bits
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


def some_ids(B, N, K, seed, kind="mixed"):
    g = gen(seed)
    if kind == "one":
        ids = torch.full((B, N), K // 2)
    elif kind == "zipf":
        w = torch.arange(1, K + 1, dtype=torch.float64).pow(-1.1)
        ids = torch.multinomial(w, B * N, replacement=True, generator=g).view(B, N)
    elif kind == "none":
        ids = torch.full((B, N), -1)
    elif kind == "once":
        ids = torch.stack([torch.randperm(K, generator=g)[:N] for _ in range(B)])
    else:
        ids = torch.randint(0, K, (B, N), generator=g)
        if N > 4:
            bad = torch.tensor([-1, K, K + 7, -(1 << 31), (1 << 31) - 1])
            at = torch.randint(0, N, (B, max(1, N // 5)), generator=g)
            ids.scatter_(1, at, bad[torch.randint(0, 5, at.shape, generator=g)])
    return ids.to(torch.int32)


def squeeze(B, *ts):
    return [t[0].contiguous() if B == 1 else t for t in ts]


# ---- lookup -------------------------------------------------------------------------------------------------------

def embed_ref(table, ids, scale, out_dtype):
    """The lookup's two roundings: fp32 product, output type.  table [B,K,D], ids [B,N], on the CPU."""
    B, K, D = table.shape
    out = torch.zeros(*ids.shape, D, dtype=F32)
    for b in range(B):
        hit = ((ids[b] >= 0) & (ids[b] < K)).nonzero()[:, 0]
        out[b, hit] = table[b, ids[b, hit].long()].float() * torch.tensor(scale, dtype=F32)
    return out.to(out_dtype)


def same(a, b):
    return torch.equal(torch.nan_to_num(a.float(), nan=12345.0, posinf=1e38, neginf=-1e38),
                       torch.nan_to_num(b.float(), nan=12345.0, posinf=1e38, neginf=-1e38))


@pytest.mark.parametrize("to", TYPES)
@pytest.mark.parametrize("of", TYPES)
@pytest.mark.parametrize("B, N, K, D", [(1, 1, 1, 1), (1, 5, 3, 80), (1, 1000, 77, 128), (3, 129, 50, 12),
                                        (2, 33, 700, 1027), (1, 7, 11, 8200), (1, 3, 5, 1026), (5, 1, 9, 16),
                                        (1, 4097, 2, 4)])
def test_embed(km, of, to, B, N, K, D):
    table = torch.randn(B, K, D, generator=gen(D)).to(of)
    ids = some_ids(B, N, K, N)
    for scale in (1.0, math.sqrt(D)):
        want = embed_ref(table, ids, scale, to)
        t, i, w = squeeze(B, table, ids, want)
        got = km.embed(t.cuda(), i.cuda(), scale=scale, out_dtype=to)
        assert got.dtype == to and got.shape == w.shape
        assert same(got.cpu(), w)


def test_embed_keeps_infinities_nan_and_subnormals(km):
    for dt in TYPES:
        fi = torch.finfo(dt)
        row = torch.tensor([math.inf, -math.inf, math.nan, fi.max, fi.min, fi.tiny, fi.tiny / 4, -0.0], dtype=dt)
        table = torch.stack([row, torch.full_like(row, math.nan)])
        ids = torch.tensor([0, -1, 1, 2], dtype=torch.int32)
        for to in TYPES:
            got = km.embed(table.cuda(), ids.cuda(), out_dtype=to).cpu()
            assert same(got, embed_ref(table[None], ids[None], 1.0, to)[0]), (dt, to)
            assert not got[1].any() and not got[3].any()      # rows of ids outside the table are zeros, whatever it holds


@pytest.mark.parametrize("D", [8, 9, 64])
def test_embed_of_slices_at_odd_addresses(km, D):
    for dt in TYPES:
        for off in (1, 2, 4):
            flat = torch.randn(off + 20 * D, generator=gen(off)).to(dt)
            buf = flat.cuda()
            table = buf[off:].view(20, D)
            ids = some_ids(1, 31, 20, off)[0]
            raw = torch.zeros(off + 31 * D, dtype=dt, device="cuda")
            out = raw[off:].view(31, D)
            assert km.embed(table, ids.cuda(), out=out) is out
            assert same(out.cpu(), embed_ref(flat[off:].view(1, 20, D), ids[None], 1.0, dt)[0])
            assert not raw[:off].any()


def test_embed_offsets_past_32_bits(km):
    # 2^31 + elements on both sides; whole rows are compared on the GPU
    K, D = (1 << 18) + 11, 8208
    table = torch.empty(K, D, dtype=BF16, device="cuda")
    table.copy_((torch.arange(K, device="cuda") % 251).to(BF16)[:, None].expand(K, D))
    ids = torch.tensor([0, K - 1, K - 7, 1 << 17, K], dtype=torch.int32, device="cuda")
    got = km.embed(table, ids)
    want = torch.tensor([0, (K - 1) % 251, (K - 7) % 251, (1 << 17) % 251, 0], device="cuda").to(BF16)
    assert torch.equal(got, want[:, None].expand(5, D))
    del table, got
    small = torch.randn(4, D, device="cuda").to(BF16)
    many = torch.arange(K, device="cuda", dtype=torch.int32) % 4
    got = km.embed(small, many)
    assert torch.equal(got[-8:], small[many[-8:].long()]) and torch.equal(got[:8], small[many[:8].long()])
    assert torch.equal(got[K // 2:K // 2 + 8], small[many[K // 2:K // 2 + 8].long()])


# ---- gradient of the lookup -------------------------------------------------------------------------------------------

def check_grad(got, dout, ids, K, scale, old=None):
    """got [B,K,D] against the definition in 64 bits; dout [B,N,D], ids [B,N], old [B,K,D] or None, on the CPU."""
    B, N, D = dout.shape
    got = got.cpu()
    s32 = float(torch.tensor(scale, dtype=F32))
    for b in range(B):
        hit = ((ids[b] >= 0) & (ids[b] < K)).nonzero()[:, 0]
        key = ids[b, hit].long()
        x = dout[b, hit].double()
        total, mag = torch.zeros(K, D, dtype=torch.float64), torch.zeros(K, D, dtype=torch.float64)
        total.index_add_(0, key, x)
        mag.index_add_(0, key, x.abs())
        m = torch.bincount(key, minlength=K).double()[:, None]
        want = s32 * total
        tol = (m + 1) * U * abs(s32) * mag * 1.01
        if old is not None:
            want = want + old[b].double()
            tol = tol + 2 * U * (want.abs() + abs(s32) * mag)
            bare = (m == 0)[:, 0]
            assert torch.equal(got[b][bare], old[b][bare])       # untouched, bit for bit
        else:
            assert not got[b][(m == 0)[:, 0]].any()
        tol = tol + (half_step(got.dtype) if got.dtype != F32 else U) * (want.abs() + tol) + tiny(got.dtype)
        bad = (got[b].double() - want).abs() > tol
        assert not bad.any(), (b, int(bad.sum()), float((got[b].double() - want).abs().max()))


GRAD_SHAPES = [(1, 1, 1, 1, "mixed"), (1, 37, 1000, 80, "mixed"), (1, 1000, 77, 128, "mixed"), (3, 129, 50, 12, "mixed"),
               (2, 333, 70, 1027, "zipf"), (1, 70, 11, 8200, "mixed"), (5, 1, 9, 16, "mixed"), (1, 5000, 300, 64, "zipf"),
               (1, 2049, 40, 256, "one"), (1, 65, 3, 24, "none"), (1, 500, 700, 32, "once"), (7, 300, 256, 16, "zipf"),
               (2, 20000, 3, 8, "one"), (1, 70001, 5000, 20, "zipf"), (1, 17000, 70000, 8, "zipf"), (64, 40, 256, 32, "mixed"),
               # one word cannot hold key and row (sorted by launches); just past each limit of the one-workgroup sorts
               (1, 9000, 300000, 8, "zipf"), (1, 257, 33, 40, "zipf"), (2, 513, 40, 136, "mixed"), (1, 4097, 131072, 4, "mixed"),
               (1, 8193, 1, 8, "one"), (1, 16385, 600, 8, "mixed"), (1, 15333, 92338, 4, "mixed"),
               (1, 900, 200000, 4, "mixed"), (1, 2000, 300, 4, "mixed"), (3, 1000, 90000, 4, "mixed"),
               # ids outside the table on every path of the sort by launches: two packed passes, three passes, one
               # segmented pass, large tiles
               (1, 70003, 5000, 20, "mixed"), (1, 70003, 300000, 4, "mixed"), (40, 2000, 200, 8, "mixed"),
               (1, 2100001, 5000, 4, "mixed"), (1, 2100001, 70000, 4, "mixed")]


@pytest.mark.parametrize("of, to", [(F32, F32), (BF16, F32), (F16, F32), (BF16, BF16), (F16, F16), (F32, BF16)])
@pytest.mark.parametrize("B, N, K, D, kind", GRAD_SHAPES)
def test_embed_grad(km, of, to, B, N, K, D, kind):
    dout = torch.randn(B, N, D, generator=gen(N)).to(of)
    ids = some_ids(B, N, K, K, kind)
    d, i = squeeze(B, dout, ids)
    for scale in (1.0, 0.3):
        got = km.embed_grad(d.cuda(), i.cuda(), K, scale=scale, grad_dtype=to)
        assert got.dtype == to and got.shape == ((K, D) if B == 1 else (B, K, D))
        check_grad(got.view(B, K, D), dout, ids, K, scale)
    old = torch.randn(B, K, D, generator=gen(7)).to(to)
    buf = squeeze(B, old.cuda())[0].clone()
    got = km.embed_grad(d.cuda(), i.cuda(), K, scale=0.3, out=buf, accumulate=True)
    assert got is buf
    check_grad(got.view(B, K, D), dout, ids, K, 0.3, old)


def test_embed_grad_of_no_rows(km):
    d, i = torch.empty(0, 24, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    out = torch.full((5, 24), 3.0, device="cuda")
    km.embed_grad(d, i, 5, out=out, accumulate=True)
    assert bool((out == 3).all())
    assert not km.embed_grad(d, i, 5, out=out).any()
    assert km.embed(out, i).shape == (0, 24)


def test_embed_grad_leaves_padding_out(km):
    # rows behind the last sequence hold NaN and infinities: nothing of them may reach a sum
    for dt in TYPES:
        dout = torch.randn(200, 40, generator=gen(1)).to(dt)
        dout[150:] = math.nan
        dout[170:, ::2] = math.inf
        ids = some_ids(1, 200, 30, 3, "zipf")[0]
        ids[150:] = -1
        got = km.embed_grad(dout.cuda(), ids.cuda(), 30)
        assert bool(torch.isfinite(got).all())
        check_grad(got[None], dout[None, :150], ids[None, :150], 30, 1.0)
    dout[3, 5] = math.nan                     # a NaN of a named row does reach its entry, and that one alone
    got = km.embed_grad(dout.cuda(), ids.cuda(), 30).cpu()
    bad = torch.isnan(got).nonzero()
    assert bad.tolist() == [[int(ids[3]), 5]]


@pytest.mark.parametrize("off", [1, 4])
def test_embed_grad_at_odd_addresses(km, off):
    for dt in TYPES:
        flat = torch.randn(off + 300 * 16, generator=gen(off)).to(dt)
        dout = flat.cuda()[off:].view(300, 16)
        ids = some_ids(1, 300, 20, off)[0]
        raw = torch.full((off + 20 * 16 + 3,), 7.0, device="cuda")
        out = raw[off:off + 320].view(20, 16)
        km.embed_grad(dout, ids.cuda(), 20, out=out)
        check_grad(out[None], flat[off:].view(1, 300, 16), ids[None], 20, 1.0)
        assert bool((raw[:off] == 7).all()) and bool((raw[off + 320:] == 7).all())


def test_embed_grad_is_the_same_every_time(km):
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    dout = torch.randn(300_000, 64, generator=g, device="cuda").to(BF16)
    ids = (torch.rand(300_000, generator=g, device="cuda") ** 4 * 2000).to(torch.int32)
    first = km.embed_grad(dout, ids, 2000)
    for _ in range(3):
        assert torch.equal(km.embed_grad(dout, ids, 2000), first)


def test_embed_grad_offsets_past_32_bits(km):
    K, D = (1 << 18) + 11, 8208
    ids = torch.tensor([K - 1, 3, K - 1, 1 << 17], dtype=torch.int32, device="cuda")
    dout = torch.randn(4, D, device="cuda").to(BF16)
    got = km.embed_grad(dout, ids, K, grad_dtype=BF16)
    assert torch.equal(got[K - 1], (dout[0].float() + dout[2].float()).to(BF16))
    assert torch.equal(got[3], dout[1]) and torch.equal(got[1 << 17], dout[3])
    touched = torch.zeros(K, dtype=torch.bool, device="cuda")
    touched[ids.long()] = True
    assert int((got != 0).any(1)[~touched].sum()) == 0
    del got
    big = torch.zeros(K, D, dtype=BF16, device="cuda")            # the rows past 2^31 elements
    big[-3:] = dout[:3]
    ids = torch.full((K,), -1, dtype=torch.int32, device="cuda")
    ids[-3:] = torch.tensor([2, 0, 2], dtype=torch.int32, device="cuda")
    got = km.embed_grad(big, ids, 4)
    assert torch.equal(got[2], dout[0].float() + dout[2].float()) and torch.equal(got[0], dout[1].float())
    assert not got[1].any() and not got[3].any()


def test_embed_grad_is_the_lookups_derivative(km):
    # <dout, embed(table)> is linear in the table: its difference in any direction is the product with the gradient
    g = gen(11)
    table, step = torch.randn(2, 40, 24, generator=g), torch.randn(2, 40, 24, generator=g)
    ids = some_ids(2, 100, 40, 5)
    dout = torch.randn(2, 100, 24, generator=g)
    up, down = (km.embed((table + s * step).cuda(), ids.cuda(), scale=1.5).double().cpu() for s in (0.5, -0.5))
    diff = (dout.double() * (up - down)).sum()
    by = (km.embed_grad(dout.cuda(), ids.cuda(), 40, scale=1.5).double().cpu() * step.double()).sum()
    # the two lookups round |values| <= about 10 to fp32 (4 roundings, 4800 values), the gradient sums to fp32
    assert abs(float(diff - by)) <= 8 * U * float((dout.double().abs() * (up.abs() + down.abs())).sum()) + \
        100 * U * float((dout.double().abs().sum()) * 1.5 * step.abs().max())


# ---- balance ------------------------------------------------------------------------------------------------------------

def balance_ref(logits, labels, valid):
    """The definition in 64 bits on the CPU.  logits [B,N,K], labels [B,N,S], valid [B,N] bool."""
    B, N, K = logits.shape
    S = labels.shape[-1]
    out = {k: [] for k in ("loss", "counts", "prob", "lse", "coef", "R")}
    for b in range(B):
        x = logits[b][valid[b]].double()
        T = x.shape[0]
        lse = torch.logsumexp(x, -1)
        p = torch.where(torch.isfinite(lse)[:, None], torch.softmax(x, -1), 0.0)
        lab = labels[b][valid[b]].reshape(-1).long()
        c = torch.bincount(lab[(lab >= 0) & (lab < K)], minlength=K)
        per = 1.0 / T if T else 0.0
        full = torch.full((N,), math.inf, dtype=torch.float64)
        full[valid[b]] = lse
        prob, coef = p.sum(0) * per, K / S * c.double() * per * per
        R = (x.amax(-1, keepdim=True) - x) if T else torch.zeros(1)
        R = float(R[torch.isfinite(R)].clamp(max=104).max()) if torch.isfinite(R).any() else 0.0
        for k, v in (("loss", (K / S * c.double() * per * prob).sum()), ("counts", c), ("prob", prob), ("lse", full),
                     ("coef", coef), ("R", R)):
            out[k].append(v)
    return {k: torch.tensor(v) if k == "R" else torch.stack(v) for k, v in out.items()}


def check_balance(got, logits, labels, valid):
    B, N, K = logits.shape
    loss, counts, prob, (lse, coef) = [t.cpu() if isinstance(t, torch.Tensor) else tuple(x.cpu() for x in t) for t in got]
    want = balance_ref(logits, labels, valid)
    counts, prob, coef, lse = counts.view(B, K), prob.view(B, K), coef.view(B, K), lse.view(B, N)
    assert torch.equal(counts.long(), want["counts"].long())
    depth = K / 64 + 24
    R = want["R"][:, None]
    rel = (2 * R + 8 + depth + ROWS) * U
    assert bool(((prob.double() - want["prob"]).abs() <= rel * want["prob"] + 2.0 ** -120).all())
    assert bool(((coef.double() - want["coef"]).abs() <= 2 * U * want["coef"]).all())
    assert bool(((loss.double() - want["loss"]).abs() <= (rel[:, 0] + U) * want["loss"] + 2.0 ** -120).all())
    inf = torch.isinf(want["lse"])
    assert torch.equal(lse[inf].double(), want["lse"][inf])
    # the sum's relative error is the logarithm's absolute one; the maximum, the logarithm and their sum round once each
    tol = (R + 4 + depth) * U + 3 * U * (want["lse"].abs() + math.log(K) + 1)
    assert bool(((lse.double() - want["lse"]).abs()[~inf] <= tol.expand(B, N)[~inf]).all())


BALANCE_SHAPES = [(1, 1, 1, 1), (1, 32, 8, 2), (1, 1000, 7, 1), (3, 257, 64, 4), (2, 300, 128, 8), (1, 129, 100, 3),
                  (1, 70, 1000, 1), (2, 65, 1024, 2), (1, 40, 3001, 5), (1, 9, 20000, 1), (1, 5, 70000, 2), (4, 1, 16, 6),
                  (70, 3, 12, 2), (1, 5000, 256, 2), (1, 3, 2, 9), (2, 900, 33, 2), (1, 515, 520, 1), (1, 66, 4104, 1),
                  (1, 300, 2048, 2), (1, 33, 8191, 3), (2, 70, 8200, 1), (1, 37, 12345, 2), (1, 21, 16384, 1)]


def balance_case(B, N, K, S, dtype, seed, spread=2.0):
    g = gen(seed)
    logits = (torch.randn(B, N, K, generator=g) * spread + torch.randn(B, 1, K, generator=g)).to(dtype)
    labels = some_ids(B, N * S, K, seed + 1).view(B, N, S)
    valid = torch.rand(B, N, generator=g) < 0.8
    return logits, labels, valid


def run_balance(km, logits, labels, valid, **kw):
    B, S = logits.shape[0], labels.shape[-1]
    x, l, v = squeeze(B, logits, labels, valid)
    if S == 1:
        l = l[..., 0].contiguous()
    return km.balance(x.cuda(), l.cuda(), valid=v.cuda(), **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B, N, K, S", BALANCE_SHAPES)
def test_balance(km, dtype, B, N, K, S):
    logits, labels, valid = balance_case(B, N, K, S, dtype, N + K)
    logits_nan = logits.clone()
    logits_nan[~valid] = math.nan                       # what an invalid row holds is of no consequence
    check_balance(run_balance(km, logits_nan, labels, valid), logits, labels, valid)
    x, l = squeeze(B, logits, labels)
    check_balance(km.balance(x.cuda(), l.cuda()), logits, labels, torch.ones_like(valid))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [5, 64, 1500, 40000])
def test_balance_of_extreme_logits(km, dtype, K):
    fi = torch.finfo(dtype)
    logits, labels, valid = balance_case(2, 12, K, 2, dtype, K)
    valid[:] = True
    logits[0, 0] = fi.min                               # a whole row of the type's lowest value: uniform
    logits[0, 1, 1:] = fi.min                           # one choice left
    logits[0, 2, : K // 2] = -math.inf                  # choices ruled out
    logits[0, 3] = -math.inf                            # none left: no probability
    logits[0, 4, K - 1] = fi.max                        # a certain choice
    logits[1, 5] = fi.max
    logits[1, 6, ::2] = fi.min
    logits[1, 6, 1::2] = fi.max
    check_balance(run_balance(km, logits, labels, valid), logits, labels, valid)
    logits[1, 7, K // 3] = math.nan                     # a NaN of a valid row spoils that instance's loss, no other's
    logits[0, 8, 2] = math.nan
    valid[0, 8] = False
    loss, counts, prob, (lse, coef) = run_balance(km, logits, labels, valid)
    assert bool(torch.isnan(loss[1])) and bool(torch.isfinite(loss[0])) and bool(torch.isnan(lse[1, 7]))
    assert torch.equal(counts.cpu().long(), balance_ref(torch.nan_to_num(logits), labels, valid)["counts"])
    logits[1, 7, K // 3] = math.inf
    assert bool(torch.isnan(run_balance(km, logits, labels, valid)[0][1]))


def test_balance_of_nothing_valid_and_of_no_rows(km):
    logits, labels, valid = balance_case(3, 50, 20, 2, BF16, 4)
    valid[1] = False
    got = run_balance(km, logits, labels, valid)
    check_balance(got, logits, labels, valid)
    assert float(got[0][1]) == 0 and not got[1][1].any() and not got[2][1].any() and not got[3][1][1].any()
    dx = km.balance_grad(logits.cuda(), got[3], torch.ones(3, device="cuda"))
    assert not dx[1].any()
    x = torch.empty(0, 20, device="cuda")
    loss, counts, prob, (lse, coef) = km.balance(x, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert float(loss) == 0 and not counts.any() and not prob.any() and lse.numel() == 0 and not coef.any()
    assert km.balance_grad(x, (lse, coef), loss).shape == (0, 20)


def test_balance_of_even_use_is_one(km):
    K = 96
    labels = torch.arange(K, dtype=torch.int32, device="cuda").repeat(10)
    loss, counts, prob, _ = km.balance(torch.zeros(10 * K, K, device="cuda"), labels)
    assert bool((counts == 10).all())
    assert abs(float(loss) - 1) <= (8 + K / 64 + 24 + ROWS) * U


def test_balance_is_the_same_every_time(km):
    logits, labels, valid = balance_case(2, 20000, 96, 4, BF16, 8)
    a = run_balance(km, logits, labels, valid)
    for _ in range(3):
        b = run_balance(km, logits, labels, valid)
        for x, y in zip((*a[:3], *a[3]), (*b[:3], *b[3])):
            assert torch.equal(x, y)


# ---- gradient of the balance loss -----------------------------------------------------------------------------------------

def check_balance_grad(got, logits, lse, coef, dloss):
    """got [B,N,K] against the formula in 64 bits from the same fp32 coef, on the rows of finite lse (all on the CPU)."""
    B, N, K = logits.shape
    z, c, dl = lse.double()[..., None], coef.double()[:, None], dloss.double().view(B, 1, 1)
    live = torch.isfinite(z)
    x = torch.where(live, logits.double(), 0.0)
    p = torch.where(live, torch.softmax(x, -1), 0.0)
    R = x.amax(-1, keepdim=True) - x
    R = torch.where(torch.isfinite(R), R.clamp(max=104), 0.0).amax(-1, keepdim=True)
    dot, mag = (p * c).sum(-1, keepdim=True), (p * c.abs()).sum(-1, keepdim=True)
    want = dl * p * (c - dot)
    rel = (2 * R + 8 + K / 64 + 24) * U
    tol = dl.abs() * p * ((rel + 4 * U) * (c.abs() + dot.abs()) + (rel + (K / 64 + 24) * U) * mag)
    tol = tol * 1.01 + half_step(got.dtype) * (want.abs() + tol) + tiny(got.dtype) + 2.0 ** -126 * dl.abs() * (c.abs() + mag)
    got = got.cpu().double()
    assert not got[~live.expand_as(got)].any()
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / tol).max()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B, N, K, S", BALANCE_SHAPES)
def test_balance_grad(km, dtype, B, N, K, S):
    logits, labels, valid = balance_case(B, N, K, S, dtype, N + K)
    hidden = logits.clone()
    hidden[~valid] = math.nan
    loss, counts, prob, saved = run_balance(km, hidden, labels, valid)
    dloss = torch.linspace(1000.0, 2000.0, B)
    got = km.balance_grad(squeeze(B, hidden)[0].cuda(), saved, dloss.cuda())
    assert got.dtype == dtype and got.shape == squeeze(B, logits)[0].shape
    lse, coef = (t.cpu().view(B, -1) for t in saved)
    check_balance_grad(got.view(B, N, K), logits, lse, coef, dloss)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [5, 64, 1500, 40000])
def test_balance_grad_of_extreme_logits(km, dtype, K):
    fi = torch.finfo(dtype)
    logits, labels, valid = balance_case(1, 12, K, 2, dtype, K)
    valid[:] = True
    logits[0, 0] = fi.min
    logits[0, 1, 1:] = fi.min
    logits[0, 2, : K // 2] = -math.inf
    logits[0, 3] = -math.inf
    logits[0, 4, K - 1] = fi.max
    logits[0, 5] = fi.max
    _, _, _, saved = run_balance(km, logits, labels, valid)
    got = km.balance_grad(logits[0].cuda(), saved, torch.tensor([100.0], device="cuda"))
    check_balance_grad(got[None], logits, saved[0].cpu()[None], saved[1].cpu()[None], torch.tensor([100.0]))


def test_balance_grad_is_the_losss_derivative(km):
    # central differences of the formula in 64 bits (the counts do not move with the logits)
    logits, labels, valid = balance_case(2, 7, 5, 2, F32, 3, spread=1.0)
    want = torch.zeros(2, 7, 5, dtype=torch.float64)
    h = 1e-5
    for b in range(2):
        for i in range(7):
            for k in range(5):
                d = torch.zeros(2, 7, 5, dtype=torch.float64)
                d[b, i, k] = h
                hi, lo = (balance_ref(logits.double() + s * d, labels, valid)["loss"][b] for s in (1, -1))
                want[b, i, k] = (hi - lo) / (2 * h)
    saved = run_balance(km, logits, labels, valid)[3]
    got = km.balance_grad(logits.cuda(), saved, torch.ones(2, device="cuda")).double().cpu()
    # differences: h^2 times a third derivative below 10, and 64-bit rounding over h; the kernel: fp32
    assert bool(((got - want).abs() <= 1e-9 + 1e-10 + 100 * U * want.abs().max()).all())


@pytest.mark.parametrize("off", [1, 2, 4])
def test_balance_at_odd_addresses(km, off):
    for dt in TYPES:
        for K in (16, 24, 200):
            logits, labels, valid = balance_case(1, 77, K, 2, dt, off)
            buf = torch.zeros(off + 77 * K, dtype=dt, device="cuda")
            x = buf[off:].view(77, K)
            x.copy_(logits[0])
            vb = torch.zeros(77 + off, dtype=torch.bool, device="cuda")
            v = vb[off:]
            v.copy_(valid[0])
            got = km.balance(x, labels[0].cuda(), valid=v)
            check_balance(got, logits, labels, valid)
            raw = torch.full((off + 77 * K + 5,), 3.0, dtype=dt, device="cuda")
            out = raw[off:off + 77 * K].view(77, K)
            km.balance_grad(x, got[3], torch.ones(1, device="cuda"), out=out)
            check_balance_grad(out[None], logits, got[3][0].cpu()[None], got[3][1].cpu()[None], torch.ones(1))
            assert bool((raw[:off] == 3).all()) and bool((raw[off + 77 * K:] == 3).all())


def test_balance_offsets_past_32_bits(km):
    N, K = (1 << 21) + 5, 1032                  # 2^31 + elements
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.empty(N, K, dtype=BF16, device="cuda")
    x[:] = torch.randn(K, generator=g, device="cuda").to(BF16)
    x[-2:] = torch.randn(2, K, generator=g, device="cuda").to(BF16)
    labels = torch.full((N,), 7, dtype=torch.int32, device="cuda")
    labels[-1] = 9
    loss, counts, prob, (lse, coef) = km.balance(x, labels)
    assert int(counts[7]) == N - 1 and int(counts[9]) == 1 and int(counts.sum()) == N
    z = torch.logsumexp(x[-2:].double(), -1)
    assert bool(((lse[-2:].double() - z).abs() <= 1e-5).all())
    want = (torch.softmax(x[0].double(), 0) * (N - 2) + torch.softmax(x[-2:].double(), -1).sum(0)) / N
    rel = (2 * 10 + 8 + K / 64 + 24 + ROWS) * U
    assert bool(((prob.double() - want).abs() <= rel * want).all())
    dx = km.balance_grad(x, (lse, coef), torch.full((1,), float(N), device="cuda"))
    check_balance_grad(dx[None, -2:], x[None, -2:].cpu(), lse[None, -2:].cpu(), coef[None].cpu(), torch.full((1,), float(N)))


# ---- how they are called ------------------------------------------------------------------------------------------------

def test_refusals_on_the_gpu(km):
    t = torch.zeros(6, 8, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    many, at = torch.zeros(300, 8, device="cuda"), torch.zeros(300, dtype=torch.int32, device="cuda")
    E = km.KMeansError
    for call in (lambda: km.embed(t, i.long()), lambda: km.embed(t, i[None]), lambda: km.embed(t[:, ::2], i),
                 lambda: km.embed(t.double(), i), lambda: km.embed(t, i, out=torch.zeros(3, 9, device="cuda")),
                 lambda: km.embed(t, i, out=t[:3]), lambda: km.embed(t, i.cpu()),
                 lambda: km.embed_grad(t, i, 4), lambda: km.embed_grad(t[:3], i, 0),
                 lambda: km.embed_grad(t[:3], i, 4, accumulate=True),
                 lambda: km.embed_grad(t[:3], i, 6, out=t), lambda: km.embed_grad(t[:3], i, 1 << 40),
                 lambda: km.embed_grad(many, at, 6, ws=torch.empty(8, device="cuda")),
                 lambda: km.embed_grad(many, at, 6, ws=torch.empty(1 << 20)),
                 lambda: km.balance(t, i), lambda: km.balance(t[:3], i.long()),
                 lambda: km.balance(t[:3], i, valid=i), lambda: km.balance(t[:3], i.new_empty(3, 0)),
                 lambda: km.balance_grad(t, (i, i), i),
                 lambda: km.balance_grad(t, (torch.zeros(6, device="cuda"),) * 2, i),
                 lambda: km.balance_grad(t[:3], (torch.zeros(3, device="cuda"), torch.zeros(8, device="cuda")),
                                         torch.zeros(1, device="cuda"), out=t[:3])):
        with pytest.raises(E):
            call()


def operators(km, s):
    """Each operator once on the state s; all their outputs."""
    e = km.embed(s["table"], s["ids"], scale=2.0, out_dtype=BF16, stream=s.get("stream"))
    g = km.embed_grad(s["dout"], s["ids"], 500, ws=s.get("ws"), stream=s.get("stream"))
    loss, counts, prob, saved = km.balance(s["logits"], s["labels"], valid=s["valid"], stream=s.get("stream"))
    dx = km.balance_grad(s["logits"], saved, s["dloss"], stream=s.get("stream"))
    return [e, g, loss, counts, prob, *saved, dx]


def a_state(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    ids = (torch.rand(4000, generator=g, device="cuda") ** 3 * 520 - 5).to(torch.int32)
    return {"table": r(500, 64), "ids": ids, "dout": r(4000, 64).to(BF16), "logits": r(2, 700, 48).to(F16),
            "labels": (torch.rand(2, 700, 3, generator=g, device="cuda") * 48).to(torch.int32),
            "valid": torch.rand(2, 700, generator=g, device="cuda") < 0.9,
            "dloss": torch.tensor([300.0, 500.0], device="cuda")}


def test_another_stream(km):
    s = a_state(1)
    want = [t.clone() for t in operators(km, s)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = operators(km, {**s, "stream": side})
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(side):
        got = operators(km, s)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once(km):
    states = [a_state(1), a_state(2)]
    want = [[t.clone() for t in operators(km, s)] for s in states]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k in range(2):
            got[k].append(operators(km, {**states[k], "stream": streams[k]}))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[k]))


def test_captured_and_replayed(km):
    states = [a_state(1), a_state(2), a_state(3)]
    want = [[t.clone() for t in operators(km, s)] for s in states]
    held = a_state(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        operators(km, held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = operators(km, held)
    for turn in (1, 2, 0, 1):
        for k, v in states[turn].items():
            held[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[turn])), turn
        eager = operators(km, states[2])                # the program's own work between the replays
        assert all(torch.equal(a, b) for a, b in zip(eager, want[2]))


def test_one_workspace_for_calls_in_a_row(km):
    ws = torch.empty(max(km.embed_grad_workspace_bytes(4000, 500, 64), km.balance_workspace_bytes(700, 48, 2, 3)),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)                                       # whatever it holds
    for seed in (1, 2):
        s = a_state(seed)
        want = operators(km, s)
        got = operators(km, {**s, "ws": ws})
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        b = km.balance(s["logits"], s["labels"], valid=s["valid"], ws=ws)
        assert torch.equal(b[0], want[2]) and torch.equal(b[1], want[3]) and torch.equal(b[2], want[4])


def test_a_codebooks_training_step(km):
    """Assign, look up, differentiate and balance as a codebook is trained, against 64 bits on the same labels."""
    g = gen(5)
    B, N, K, D = 2, 3000, 64, 32
    C = torch.randn(B, K, D, generator=g)
    X = (C[:, torch.randint(0, K, (N,), generator=g)] + 0.3 * torch.randn(B, N, D, generator=g)).to(BF16)
    Xg, Cg = X.cuda(), C.cuda()
    labels, _, _ = km.assign(Xg, Cg)
    q = km.embed(Cg, labels, out_dtype=F32)
    assert same(q.cpu(), embed_ref(C, labels.cpu(), 1.0, F32))
    dq = (q - Xg.float()) * (2.0 / N)                     # of the mean squared distance
    dC = km.embed_grad(dq, labels, K)
    check_grad(dC, dq.cpu(), labels.cpu(), K, 1.0)
    # two selections a row, and a softmax over the distances' scores
    labels2, _ = km.assign_top2(Xg, Cg)
    logits = (torch.stack([Xg[b].float() @ Cg[b].T for b in range(B)]) - 0.5 * (Cg * Cg).sum(-1)[:, None]).contiguous()
    got = km.balance(logits, labels2)
    check_balance(got, logits.cpu(), labels2.cpu(), torch.ones(B, N, dtype=torch.bool))
    dx = km.balance_grad(logits, got[3], torch.full((B,), 0.01 * N, device="cuda"))
    check_balance_grad(dx, logits.cpu(), got[3][0].cpu(), got[3][1].cpu(), torch.full((B,), 0.01 * N))
    # the update's counts are the balance's where one label a row is counted
    _, counts = km.update(Xg, labels, Cg)
    assert torch.equal(km.balance(logits, labels)[1], counts)
