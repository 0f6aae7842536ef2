"""Cases for the codebook operators: table lookup with scaling and its gradient by sorted ids, and the balance loss of
a router's or codebook's use with its counts and gradient.

``run`` computes a case in plain torch operations, or, where ``own`` is set, through this repository's entry points.
``exact`` computes the same outputs in 64 bits from the definitions.

Definitions (B independent instances; N rows, K table entries or choices, D columns, S selections a row):

  embed         out[b,i,:]  = scale * table[b, ids[b,i], :]                  (a zero row where the id is outside [0,K))
  embed_grad    grad[b,k,:] = old[b,k,:] + scale * sum of dout[b,i,:] over the rows i with ids[b,i] = k
                              (old is zero without accumulation)
  balance       p[b,i,:]    = softmax(logits[b,i,:]),  lse[b,i] = log sum exp of the row,  T[b] = valid rows
                prob[b,k]   = sum of p[b,i,k] over the valid rows / T[b]
                counts[b,k] = selections (b,i,s) of valid rows that name k
                loss[b]     = K * sum_k counts[b,k] / (S T[b]) * prob[b,k]
                coef[b,k]   = K * counts[b,k] / (S T[b]^2)   (the loss's derivative by each valid p[b,i,k])
                rows that are not valid leave nothing and have lse = +inf
  balance_grad  dlogits     = dloss[b] * p * (coef - sum_j p_j coef_j) a row, p = exp(logits - lse); zero where lse = +inf
"""

import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}

#: Over more rows than this the plain form takes its sums in 64 bits.
LONG = 1 << 17


def listed():
    return [
        # the newest token of each of 16 sequences: latency is all that counts
        {"name": "embed_step", "op": "embed", "B": 1, "N": 16, "K": 32000, "D": 2048, "type": "bf16", "to": "bf16",
         "scale": 1.0, "pad": 0.0},
        # one long ragged prompt, a vocabulary that is no round number, rows scaled by sqrt(D)
        {"name": "embed_prompt", "op": "embed", "B": 1, "N": 8191, "K": 50257, "D": 1600, "type": "f16", "to": "f16",
         "scale": 40.0, "pad": 0.0},
        # every point of a large clustering problem decoded to its (fp32) centroid
        {"name": "embed_codebook", "op": "embed", "B": 1, "N": 1 << 23, "K": 65536, "D": 128, "type": "f32", "to": "bf16",
         "scale": 1.0, "pad": 0.0},
        # the gradient of a small table from one short row: latency
        {"name": "grad_tiny", "op": "embed_grad", "B": 1, "N": 37, "K": 1000, "D": 80, "type": "f32", "to": "f32",
         "scale": 1.0, "pad": 0.0, "accumulate": False},
        # one training step's tokens, a tenth of them padding, Zipf-distributed ids
        {"name": "grad_tokens", "op": "embed_grad", "B": 1, "N": 16384, "K": 32000, "D": 2048, "type": "bf16",
         "to": "f32", "scale": 1.0, "pad": 0.1, "accumulate": False},
        # a later microbatch added to the gradient of a large vocabulary
        {"name": "grad_accumulate", "op": "embed_grad", "B": 1, "N": 4099, "K": 131072, "D": 1024, "type": "f16",
         "to": "f32", "scale": 32.0, "pad": 0.0, "accumulate": True},
        # the codebook's gradient from every point of a large clustering problem, hot entries among them
        {"name": "grad_codebook", "op": "embed_grad", "B": 1, "N": 1 << 23, "K": 65536, "D": 128, "type": "bf16",
         "to": "f32", "scale": 1.0, "pad": 0.0, "accumulate": False},
        # a decoding batch's router: latency
        {"name": "balance_step", "op": "balance", "B": 1, "N": 32, "K": 8, "S": 2, "type": "f32", "pad": 0.0},
        # eight sequences of a training step, each balanced by itself, 128 experts, 8 a token, padded tails
        {"name": "balance_experts", "op": "balance", "B": 8, "N": 4095, "K": 128, "S": 8, "type": "f16", "pad": 0.1},
        # the use of a codebook of 1,024 entries by a million points
        {"name": "balance_codebook", "op": "balance", "B": 1, "N": 1 << 20, "K": 1024, "S": 1, "type": "bf16", "pad": 0.0},
        # the gradients of the last two
        {"name": "balance_grad_experts", "op": "balance_grad", "B": 8, "N": 4095, "K": 128, "S": 8, "type": "bf16",
         "pad": 0.1},
        {"name": "balance_grad_codebook", "op": "balance_grad", "B": 1, "N": 1 << 20, "K": 1024, "S": 1, "type": "bf16",
         "pad": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "balance", "balance_grad"])
    kind = rng.choice(["f32", "f16", "bf16"])
    pad = rng.choice([0.0, 0.0, 0.1, 0.5])
    B = rng.choice([1, 1, 1, 2, rng.randint(3, 64)])
    if op in ("embed", "embed_grad"):
        D = rng.choice([16, 32, 64, 128, 256, _log(rng, 1, 8192), 8 * _log(rng, 2, 1024)])
        K = max(1, min(_log(rng, 1, 200000), (1 << 28) // (D * B)))
        N = max(1, min(_log(rng, 1, 1 << 22), (1 << 29) // (D * B)))
        case = {"op": op, "B": B, "N": N, "K": K, "D": D, "type": kind,
                "to": rng.choice([kind, "f32"]) if op == "embed_grad" else rng.choice([kind, kind, "bf16"]),
                "scale": rng.choice([1.0, round(math.sqrt(D), 4), 0.125]), "pad": pad}
        if op == "embed_grad":
            case["accumulate"] = case["to"] == "f32" and rng.random() < 0.4
        return case
    K = rng.choice([8, 16, 64, 128, 256, _log(rng, 1, 16384), _log(rng, 1, 1024)])
    N = max(1, min(_log(rng, 1, 1 << 20), (1 << 28) // (K * B)))
    return {"op": op, "B": B, "N": N, "K": K, "S": rng.randint(1, min(8, K)), "type": kind, "pad": pad}


# ---- inputs ------------------------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _zipf(g, B, n, K):
    """[B, n] int32 ids in [0, K), each instance's drawn from a Zipf(1.1) law over a shuffled table."""
    w = torch.arange(1, K + 1, device="cuda", dtype=torch.float64).pow(-1.1)
    cdf = torch.cumsum(w, 0)
    cdf /= cdf[-1].clone()
    u = torch.rand(B * n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.searchsorted(cdf, u).clamp_(max=K - 1)
    name = torch.randperm(K, generator=g, device="cuda")
    return name[rank].to(torch.int32).view(B, n)


def _valid(case):
    """[B, N] bool: the rows before each instance's padded tail (instances end at different rows)."""
    B, N = case["B"], case["N"]
    ends = [N - int(case["pad"] * N * 2 * (b + 1) / (B + 1)) for b in range(B)]
    return torch.arange(N, device="cuda")[None, :] < torch.tensor(ends, device="cuda")[:, None]


def _normal(g, shape, kind, spread=1.0):
    """Normal values of the type; large tensors in pieces, so that no 32-bit copy of them is made."""
    out = torch.empty(shape, dtype=TYPES[kind], device="cuda")
    flat, piece = out.view(-1), 1 << 27
    for at in range(0, flat.numel(), piece):
        n = min(piece, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=g, device="cuda") * spread
    return out


def _squeeze(case, t):
    return t[0] if case["B"] == 1 and t is not None else t


def prepare(case, seed):
    g = _generator(seed)
    B, N, K = case["B"], case["N"], case["K"]
    valid = _valid(case)
    s = {"case": case}
    if case["op"] in ("embed", "embed_grad"):
        D = case["D"]
        ids = _zipf(g, B, N, K)
        s["ids"] = _squeeze(case, torch.where(valid, ids, torch.full_like(ids, -1)))
        if case["op"] == "embed":
            s["table"] = _squeeze(case, _normal(g, (B, K, D), case["type"], 0.02 if case["scale"] != 1.0 else 1.0))
        else:
            s["dout"] = _squeeze(case, _normal(g, (B, N, D), case["type"], 0.1))
            if case["accumulate"]:
                s["grad"] = _squeeze(case, _normal(g, (B, K, D), case["to"]))
        return s
    # a router's scores: a preference a choice has for every row, and each row's own taste
    logits = _normal(g, (B, N, K), case["type"], 1.5)
    logits += torch.randn((B, 1, K), generator=g, device="cuda").to(logits.dtype)
    s["logits"] = _squeeze(case, logits)
    if case["op"] == "balance":
        S = case["S"]
        labels = torch.topk(logits.view(B * N, K), S, dim=-1).indices.to(torch.int32).view(B, N, S)
        s["labels"] = _squeeze(case, labels if S > 1 else labels[..., 0].contiguous())
        s["valid"] = _squeeze(case, valid) if case["pad"] else None
        return s
    # what the forward pass leaves for the backward pass
    lse = torch.logsumexp(logits.float(), -1)
    s["lse"] = _squeeze(case, torch.where(valid, lse, torch.full_like(lse, math.inf)))
    T = valid.sum(1, keepdim=True).clamp_(min=1).double()
    share = torch.rand((B, K), generator=g, device="cuda", dtype=torch.float64) ** 2
    share /= share.sum(1, keepdim=True)
    counts = (share * T * case["S"]).round()
    s["coef"] = _squeeze(case, (counts * (K / case["S"]) / (T * T)).float())
    # the loss's weight, scaled so that the gradients stay in the type's range
    s["dloss"] = torch.full((B,), 0.01 * 65536.0, device="cuda")
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"embed": _embed, "embed_grad": _embed_grad, "balance": _balance, "balance_grad": _balance_grad}[
        state["case"]["op"]](state)


def _own(s):
    import exact_means_clustering_amd as km

    c = s["case"]
    if c["op"] == "embed":
        return km.embed(s["table"], s["ids"], scale=c["scale"], out_dtype=TYPES[c["to"]])
    if c["op"] == "embed_grad":
        if c["accumulate"]:
            return km.embed_grad(s["dout"], s["ids"], c["K"], scale=c["scale"], out=s["grad"], accumulate=True)
        return km.embed_grad(s["dout"], s["ids"], c["K"], scale=c["scale"], grad_dtype=TYPES[c["to"]])
    if c["op"] == "balance":
        loss, counts, prob, (lse, coef) = km.balance(s["logits"], s["labels"], valid=s["valid"])
        return {"loss": loss, "counts": counts, "prob": prob, "lse": lse, "coef": coef}
    return km.balance_grad(s["logits"], (s["lse"], s["coef"]), s["dloss"])


def _flat(ids, B, K):
    """Ids as rows of the B tables laid end to end, and the row past them for ids outside [0, K)."""
    ids = ids.view(B, -1).long()
    base = torch.arange(B, device=ids.device)[:, None] * K
    return torch.where((ids >= 0) & (ids < K), ids + base, B * K).view(-1)


def _embed(s):
    c = s["case"]
    B, K, D = c["B"], c["K"], c["D"]
    at = _flat(s["ids"], B, K)
    rows = s["table"].view(B * K, D)[at.clamp(max=B * K - 1)].float() * c["scale"]
    rows = torch.where((at < B * K)[:, None], rows, 0.0)
    return rows.to(TYPES[c["to"]]).view(*s["ids"].shape, D)


def _embed_grad(s):
    c = s["case"]
    B, K, D = c["B"], c["K"], c["D"]
    at, dout = _flat(s["ids"], B, K), s["dout"].view(-1, D)
    if c["N"] > LONG:
        # running sums over the rows in the order of their ids, and their differences at the ends of each id's run
        at, order = torch.sort(at, stable=True)
        ends = torch.searchsorted(at, torch.arange(B * K + 1, device="cuda"), right=True)
        sums = torch.zeros((D, at.numel() + 1), dtype=torch.float64, device="cuda")
        sums[:, 1:] = torch.cumsum(dout[order].t().contiguous(), 1, dtype=torch.float64)
        sums = sums[:, ends].t()
        total = torch.cat((sums[:1], sums[1:] - sums[:-1]))
    else:
        total = torch.zeros((B * K + 1, D), device="cuda")
        total.index_add_(0, at, dout.float())
    total = total[:-1].mul_(c["scale"]).view(*((B, K, D) if B > 1 else (K, D)))
    if c["accumulate"]:
        s["grad"].copy_(total.add_(s["grad"]))
        return s["grad"]
    return total.to(TYPES[c["to"]])


def _balance(s):
    c = s["case"]
    B, N, K, S = c["B"], c["N"], c["K"], c["S"]
    logits = s["logits"].view(B, N, K).float()
    valid = s["valid"].view(B, N) if s["valid"] is not None else torch.ones((B, N), dtype=torch.bool, device="cuda")
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    live = valid[..., None] & (top > -math.inf)
    lse = torch.where(valid, (top + total.log())[..., 0], math.inf)
    T = valid.sum(1).double()[:, None]
    per = torch.where(T > 0, 1.0 / T, 0.0)
    prob = torch.where(live, e / total, 0.0).sum(1, dtype=torch.float64) * per
    at = torch.where(valid[..., None], s["labels"].view(B, N, S), -1)
    counts = torch.zeros(B * K + 1, dtype=torch.int32, device="cuda")
    counts.index_add_(0, _flat(at, B, K), torch.ones(B * N * S, dtype=torch.int32, device="cuda"))
    counts = counts[:-1].view(B, K)
    share = counts.double() * (per * (K / S))
    shape = (B, K) if B > 1 else (K,)
    return {"loss": (share * prob).sum(1).float(), "counts": counts.view(shape), "prob": prob.float().view(shape),
            "lse": lse.view(s["logits"].shape[:-1]), "coef": (share * per).float().view(shape)}


def _balance_grad(s):
    c = s["case"]
    B, N, K = c["B"], c["N"], c["K"]
    logits, lse = s["logits"].view(B, N, K).float(), s["lse"].view(B, N, 1)
    coef = s["coef"].view(B, 1, K)
    p = torch.where(torch.isfinite(lse), torch.exp(logits - lse), 0.0)
    d = s["dloss"].view(B, 1, 1) * p * (coef - (p * coef).sum(-1, keepdim=True))
    return d.to(s["logits"].dtype).view(s["logits"].shape)


# ---- the least a pass moves and computes ---------------------------------------------------------------------------------

def work(case):
    B, N, K = case["B"], case["N"], case["K"]
    e = BYTES[case["type"]]
    if case["op"] in ("embed", "embed_grad"):
        D, live = case["D"], N - int(case["pad"] * N)
        touched = min(K, live)
        if case["op"] == "embed":
            return {"bytes": B * (4 * N + touched * D * e + N * D * BYTES[case["to"]]), "flops": B * N * D}
        entries = 2 * touched if case["accumulate"] else K
        return {"bytes": B * (4 * N + live * D * e + entries * D * BYTES[case["to"]]), "flops": B * live * D}
    live = N - int(case["pad"] * N)
    if case["op"] == "balance":
        return {"bytes": B * (live * (K * e + 4 * case["S"]) + 4 * N + 12 * K), "flops": 5 * B * live * K}
    return {"bytes": B * ((live + N) * K * e + 4 * N + 4 * K), "flops": 7 * B * live * K}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    B, N, K = case["B"], case["N"], case["K"]
    if case["op"] in ("embed", "embed_grad"):
        D, ids = case["D"], s["ids"].reshape(B, N).long()
        if case["op"] == "embed":
            out = torch.zeros((B, N, D), dtype=torch.float64, device="cuda")
            for b in range(B):
                hit = ((ids[b] >= 0) & (ids[b] < K)).nonzero()[:, 0]
                out[b, hit] = s["table"].reshape(B, K, D)[b].index_select(0, ids[b, hit]).double() * case["scale"]
            return out.view(*s["ids"].shape, D)
        grad = torch.zeros((B, K, D), dtype=torch.float64, device="cuda")
        for b in range(B):
            order = torch.argsort(ids[b], stable=True)
            order = order[ids[b, order] >= 0]
            have, many = torch.unique_consecutive(ids[b, order], return_counts=True)
            if have.numel():
                rows = s["dout"].reshape(B, N, D)[b, order].double()
                grad[b, have] = torch.segment_reduce(rows, "sum", lengths=many, axis=0) * case["scale"]
        grad = grad if B > 1 else grad[0]
        return grad + s["grad"].double() if case["accumulate"] else grad
    logits = s["logits"].reshape(B, N, K).double()
    if case["op"] == "balance":
        S = case["S"]
        valid = s["valid"].reshape(B, N) if s["valid"] is not None else torch.ones((B, N), dtype=torch.bool, device="cuda")
        labels = s["labels"].reshape(B, N, S).long()
        out = {"loss": [], "counts": [], "prob": [], "lse": [], "coef": []}
        for b in range(B):
            rows = logits[b][valid[b]]
            T = max(1, rows.shape[0])
            p = torch.softmax(rows, -1)
            prob = p.sum(0) / T
            named = torch.bincount(labels[b][valid[b]].reshape(-1), minlength=K).double()
            lse = torch.full((N,), math.inf, dtype=torch.float64, device="cuda")
            lse[valid[b]] = torch.logsumexp(rows, -1)
            for name, v in (("loss", K * (named / (S * T) * prob).sum()), ("counts", named), ("prob", prob), ("lse", lse),
                            ("coef", K * named / (S * T) / T)):
                out[name].append(v)
        got = {name: torch.stack(v) for name, v in out.items()}
        got["counts"] = None
        return {name: v if v is None or B > 1 or name == "loss" else v[0] for name, v in got.items()}
    lse = s["lse"].reshape(B, N, 1).double()
    p = torch.exp(logits - lse)
    coef = s["coef"].reshape(B, 1, K).double()
    mean = torch.matmul(p, coef.transpose(1, 2).contiguous())
    return (p * (coef - mean) * s["dloss"].double().view(B, 1, 1)).view(s["logits"].shape)
