"""Cases for the operators of a router's and a codebook's training step: routing to choices (scores, a bias for balance,
groups, top-k, weights) with its gradient, and the AdamW step over many tensors with states in 32 bits or in 8.

``run`` computes a case in plain torch operations, or, where ``own`` is set, through this repository's entry points.
``exact`` computes the same outputs in 64 bits from the definitions.

Definitions (N rows of B instances, K choices, S selections a row, G groups of K / G neighbouring choices):

  route       s = softmax(logits) or sigmoid(logits) a row,  c = s + bias  (-inf where the logit is -inf)
              with G > 1: a group's score is the sum of its `best` (1 or 2) largest c; the `keep` groups of the highest
              score stay, the others' choices are out
              ids     = the S choices of the largest c in descending order, ties to the lowest index; -1 where none is left
              chosen  = the logits of the ids (-inf for an id of -1)
              weights = scale * s[ids], or scale * s[ids] / sum s[ids] (renormalised); 0 for an id of -1
              a row that is not valid has no choices
  route_grad  dlogits = the derivative of sum(weights * dweights) with respect to the logits, the ids held fixed; added to
              an old gradient with accumulation
  adamw       g = grad,  m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g g
              p' = p (1 - lr wd) - lr / (1 - b1^t) * m' / (sqrt(v' / (1 - b2^t)) + eps)
              p is the master copy where there is one, and the parameter its rounding.
              In 8 bits m and v are float8 (e4m3 and e5m2) times a factor per 256 values of a tensor, which is the largest
              magnitude among them / 2^8 and / 2^15; a positive v is at least the type's smallest value (2^-16); the step
              uses m' and v' before they are rounded.
"""

import math
import random

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 256  # values that share a factor


def listed():
    return [
        # a decoding batch's router: latency is all that counts
        {"name": "route_step", "op": "route", "B": 1, "N": 8, "K": 256, "S": 8, "type": "f32", "score": "sigmoid",
         "bias": True, "G": 8, "keep": 4, "best": 2, "renorm": True, "scale": 2.5, "pad": 0.0, "masked": 0.0},
        # few large experts, two a token, four ragged sequences
        {"name": "route_few", "op": "route", "B": 4, "N": 4095, "K": 8, "S": 2, "type": "f16", "score": "softmax",
         "bias": False, "G": 1, "keep": 1, "best": 1, "renorm": True, "scale": 1.0, "pad": 0.1, "masked": 0.0},
        # a training step's tokens over 128 experts, 8 a token
        {"name": "route_experts", "op": "route", "B": 1, "N": 32768, "K": 128, "S": 8, "type": "bf16", "score": "softmax",
         "bias": False, "G": 1, "keep": 1, "best": 1, "renorm": True, "scale": 1.0, "pad": 0.0, "masked": 0.0},
        # many small experts in groups, balanced by a bias
        {"name": "route_groups", "op": "route", "B": 1, "N": 65536, "K": 256, "S": 8, "type": "f32", "score": "sigmoid",
         "bias": True, "G": 8, "keep": 4, "best": 2, "renorm": True, "scale": 2.5, "pad": 0.0, "masked": 0.0},
        # two entries of a codebook of 1,024 for each of many points, weighted by their probabilities
        {"name": "route_codebook", "op": "route", "B": 1, "N": 1 << 18, "K": 1024, "S": 2, "type": "bf16",
         "score": "softmax", "bias": False, "G": 1, "keep": 1, "best": 1, "renorm": False, "scale": 1.0, "pad": 0.0,
         "masked": 0.0},
        # the gradients: eight sequences with padded tails; onto the balance loss's gradient; of the probabilities themselves
        {"name": "route_grad_experts", "op": "route_grad", "B": 8, "N": 4095, "K": 128, "S": 8, "type": "bf16",
         "score": "softmax", "renorm": True, "scale": 1.0, "pad": 0.1, "masked": 0.0, "accumulate": False},
        {"name": "route_grad_onto", "op": "route_grad", "B": 1, "N": 65536, "K": 256, "S": 8, "type": "f32",
         "score": "sigmoid", "renorm": True, "scale": 2.5, "pad": 0.0, "masked": 0.0, "accumulate": True},
        {"name": "route_grad_codebook", "op": "route_grad", "B": 1, "N": 1 << 18, "K": 1024, "S": 2, "type": "bf16",
         "score": "softmax", "renorm": False, "scale": 1.0, "pad": 0.0, "masked": 0.0, "accumulate": False},
        # a router, its norms and a small table: latency
        {"name": "adamw_router", "op": "adamw", "count": 7, "total": 60000, "type": "f32", "grad": "f32", "master": False,
         "bits": 32},
        # a codebook of 65,536 entries of 128 values
        {"name": "adamw_codebook", "op": "adamw", "count": 1, "total": 65536 * 128, "type": "f32", "grad": "f32",
         "master": False, "bits": 32},
        # a small model's tensors in bf16 with fp32 master copies
        {"name": "adamw_model", "op": "adamw", "count": 148, "total": 124000000, "type": "bf16", "grad": "bf16",
         "master": True, "bits": 32},
        # a larger one's, with states in 8 bits
        {"name": "adamw_model_8bit", "op": "adamw", "count": 290, "total": 350000000, "type": "bf16", "grad": "bf16",
         "master": True, "bits": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "adamw"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "adamw":
        bits = rng.choice([8, 32])
        total = _log(rng, 1, 1 << 27)
        return {"op": op, "count": min(total, _log(rng, 1, 300)), "total": total, "type": kind,
                "grad": rng.choice([kind, kind, "f32"]), "master": kind != "f32" and rng.random() < 0.6, "bits": bits}
    pad, masked = rng.choice([0.0, 0.0, 0.1, 0.5]), rng.choice([0.0, 0.0, 0.2])
    B = rng.choice([1, 1, 1, 2, rng.randint(3, 32)])
    K = rng.choice([8, 64, 128, 160, 256, _log(rng, 2, 2048), _log(rng, 2, 512)])
    S = min(K, rng.choice([1, 2, 4, 6, 8, 8, rng.randint(1, 16)]))
    N = max(1, min(_log(rng, 1, 1 << 20), (1 << 26) // (K * B)))
    case = {"op": op, "B": B, "N": N, "K": K, "S": S, "type": kind, "score": rng.choice(["softmax", "sigmoid"]),
            "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5, 16.0]), "pad": pad, "masked": masked}
    if op == "route_grad":
        return {**case, "accumulate": rng.random() < 0.4}
    divisors = [g for g in range(2, 33) if K % g == 0 and K // g >= 2]
    G = rng.choice(divisors) if divisors and rng.random() < 0.5 else 1
    least = -(-S * G // K)  # groups that hold S choices
    return {**case, "bias": rng.random() < 0.5, "G": G, "keep": rng.randint(least, G), "best": rng.choice([1, 2])}


# ---- inputs ------------------------------------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _normal(g, shape, kind, spread=1.0):
    """Normal values of the type; large tensors in pieces, so that no 32-bit copy of them is made."""
    out = torch.empty(shape, dtype=TYPES[kind], device="cuda")
    flat, piece = out.view(-1), 1 << 26
    for at in range(0, flat.numel(), piece):
        n = min(piece, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=g, device="cuda") * spread
    return out


def _squeeze(case, t):
    return t[0] if case["B"] == 1 and t is not None else t


def _valid(case):
    """[B, N] bool: the rows before each instance's padded tail (instances end at different rows)."""
    B, N = case["B"], case["N"]
    ends = [N - int(case["pad"] * N * 2 * (b + 1) / (B + 1)) for b in range(B)]
    return torch.arange(N, device="cuda")[None, :] < torch.tensor(ends, device="cuda")[:, None]


def sizes(case):
    """The tensors' numbers of elements: a few large ones, many small ones, hardly any a round number."""
    count, total = case["count"], case["total"]
    if count == 1:
        return [total]
    r = random.Random(1000003 * count + total)
    share = [math.exp(r.gauss(0.0, 2.0)) for _ in range(count)]
    left = total - count
    got = [1 + int(left * x / sum(share)) for x in share]
    got[0] += total - sum(got)
    return got


def prepare(case, seed):
    g = _generator(seed)
    return _prepare_adamw(case, g) if case["op"] == "adamw" else _prepare_route(case, g)


def _prepare_route(case, g):
    B, N, K, S = case["B"], case["N"], case["K"], case["S"]
    valid = _valid(case)
    s = {"case": case, "valid": _squeeze(case, valid) if case["pad"] else None, "bias": None}
    # a router's scores: a preference a choice has for every row, and each row's own taste; some choices out of use
    logits = _normal(g, (B, N, K), case["type"], 1.5)
    logits += torch.randn((B, 1, K), generator=g, device="cuda").to(logits.dtype)
    if case["masked"]:
        logits.masked_fill_(torch.rand((B, 1, K), generator=g, device="cuda") < case["masked"], -math.inf)
    s["logits"] = _squeeze(case, logits)
    if case["op"] == "route":
        if case["bias"]:
            # moved by a thousandth a step, up or down
            s["bias"] = torch.randint(-40, 41, (K,), generator=g, device="cuda").float() * 0.001
        return s
    # what the forward pass leaves for the backward pass
    val, ids = torch.topk(logits.view(B * N, K), S, dim=-1)
    live = valid.view(-1, 1) & (val > -math.inf)
    s["ids"] = _squeeze(case, torch.where(live, ids, -1).to(torch.int32).view(B, N, S))
    s["chosen"] = _squeeze(case, torch.where(live, val.float(), -math.inf).view(B, N, S))
    s["dweights"] = _squeeze(case, torch.randn((B, N, S), generator=g, device="cuda"))
    if case["accumulate"]:
        s["grad"] = _squeeze(case, _normal(g, (B, N, K), case["type"], 0.1))
    return s


def _prepare_adamw(case, g):
    """Every tensor starts on a whole block of flat buffers, as a program that keeps its parameters in one piece has them;
    what is between two tensors is zero and stays so."""
    each = sizes(case)
    starts, end = [], 0
    for n in each:
        starts.append(end)
        end += -(-n // BLOCK) * BLOCK
    blocks = end // BLOCK
    # gradients of different tensors and of parts of them differ by orders of magnitude
    size = torch.exp(torch.randn((blocks, 1), generator=g, device="cuda") * 2.0 - 6.0)
    live = torch.zeros(end, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, each):
        live[a:a + n] = True
    flat = lambda t, kind: torch.where(live, t.view(-1), 0.0).to(TYPES[kind])  # noqa: E731
    normal = lambda: torch.randn((blocks, BLOCK), generator=g, device="cuda")  # noqa: E731
    p = flat(normal() * 0.1, "f32")
    s = {"case": case, "p": p.to(TYPES[case["type"]]), "master": p if case["master"] else None}
    s["g"] = flat(normal() * size, case["grad"])
    s["m"] = flat(normal() * size * 0.3, "f32")
    s["v"] = flat(normal().square() * size * size + 1e-3 * size * size, "f32")
    s["sm"] = s["sv"] = None
    if case["bits"] == 8:
        s["m"], s["sm"] = _to_8bit(s["m"], torch.float8_e4m3fn, 256.0, 0.0)
        s["v"], s["sv"] = _to_8bit(s["v"], torch.float8_e5m2, 32768.0, 2.0 ** -16)
    s["rate"] = {"lr": 1e-4, "step": 1000, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1}
    if own:
        import exact_means_clustering_amd as km

        part = lambda t: None if t is None else [t[a:a + n] for a, n in zip(starts, each)]  # noqa: E731
        scale = lambda t: [t[a // BLOCK:a // BLOCK + -(-n // BLOCK)] for a, n in zip(starts, each)]  # noqa: E731
        s["plan"] = km.adamw_plan(part(s["p"]), part(s["g"]), part(s["m"]), part(s["v"]), masters=part(s["master"]),
                                  scales=(scale(s["sm"]), scale(s["sv"])) if case["bits"] == 8 else None)
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"route": _route, "route_grad": _route_grad, "adamw": _adamw}[state["case"]["op"]](state)


def _own(s):
    import exact_means_clustering_amd as km

    c = s["case"]
    if c["op"] == "route":
        ids, weights, chosen = km.route(s["logits"], c["S"], score=c["score"], bias=s["bias"], groups=c["G"],
                                        top_groups=c["keep"], group_best=c["best"], renormalise=c["renorm"],
                                        scale=c["scale"], valid=s["valid"])
        return {"ids": ids, "weights": weights, "chosen": chosen}
    if c["op"] == "route_grad":
        return km.route_grad(s["logits"], s["ids"], s["chosen"], s["dweights"], score=c["score"], renormalise=c["renorm"],
                             scale=c["scale"], out=s.get("grad"), accumulate=c["accumulate"])
    km.adamw(s["plan"], **s["rate"])
    return _outputs(s)


def _route(s):
    c = s["case"]
    K, S, G = c["K"], c["S"], c["G"]
    x = s["logits"].view(-1, K)
    softmax, best = c["score"] == "softmax", min(c["best"], K // G)
    # the order of the scores is the logits' own, unless they are added to something: then it is taken in 64 bits
    key = x.float()
    if c["bias"] or (G > 1 and best == 2):
        key = x.double()
        if softmax:
            key = torch.exp(key - key.amax(-1, keepdim=True))
            key = key / key.sum(-1, keepdim=True)
        else:
            key = 1.0 / (1.0 + torch.exp(-key))
        if c["bias"]:
            key = key + s["bias"].double()
        key = torch.where(x > -math.inf, key, -math.inf)
    if G > 1:
        per = key.view(-1, G, K // G)
        top = torch.sort(per, dim=-1, descending=True).values[..., :best]
        score = torch.where(top > -math.inf, top, 0.0).sum(-1)
        score = torch.where(top[..., 0] > -math.inf, score, -math.inf)
        order = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros(score.shape, dtype=torch.bool, device="cuda").scatter_(1, order, True)
        key = torch.where(keep[..., None], per, -math.inf).view(-1, K)
    top, ids = torch.sort(key, dim=-1, descending=True, stable=True)
    ids, live = ids[:, :S], top[:, :S] > -math.inf
    if s["valid"] is not None:
        live = live & s["valid"].view(-1, 1)
    chosen = torch.where(live, x.gather(1, ids).float(), -math.inf)
    if softmax and not c["renorm"]:
        high = x.amax(-1, keepdim=True).float()
        w = torch.exp(chosen - high) / torch.exp(x.float() - high).sum(-1, keepdim=True)
    else:
        w = _shares(chosen, softmax, c["renorm"])
    w = torch.where(live, w * c["scale"], 0.0)
    shape = (*s["logits"].shape[:-1], S)
    return {"ids": torch.where(live, ids, -1).to(torch.int32).view(shape), "weights": w.view(shape),
            "chosen": chosen.view(shape)}


def _shares(chosen, softmax, renorm):
    """The scores of the chosen logits, or their shares of the row's sum (taken relative to the largest)."""
    if not renorm:
        return 1.0 / (1.0 + torch.exp(-chosen))
    high = chosen.amax(-1, keepdim=True)
    high = torch.where(high > -math.inf, high if softmax else high.clamp(max=0.0), 0.0)
    e = torch.exp(chosen - high)
    if not softmax:
        e = torch.where(chosen > 0.0, 1.0 / (1.0 + torch.exp(-chosen)), e / (1.0 + torch.exp(chosen)))
    return e / e.sum(-1, keepdim=True)


def _route_grad(s):
    c = s["case"]
    K, S, softmax = c["K"], c["S"], c["score"] == "softmax"
    ids, z, dw = s["ids"].view(-1, S).long(), s["chosen"].view(-1, S), s["dweights"].view(-1, S) * c["scale"]
    live = ids >= 0
    dw = torch.where(live, dw, 0.0)
    at = torch.where(live, ids, K)
    wide = torch.zeros((ids.shape[0], K + 1), device="cuda")
    if softmax and not c["renorm"]:
        wide.scatter_add_(1, at, dw)
        x = s["logits"].view(-1, K).float()
        e = torch.exp(x - x.amax(-1, keepdim=True))
        p = torch.where(live.any(-1, keepdim=True), e / e.sum(-1, keepdim=True), 0.0)
        d = wide[:, :K]
        d = p * (d - (p * d).sum(-1, keepdim=True))
    else:
        w = torch.where(live, _shares(z, softmax, c["renorm"]), 0.0)
        d = w * (dw - (w * dw).sum(-1, keepdim=True)) if c["renorm"] else w * dw
        if not softmax:
            d = torch.where(live, d / (1.0 + torch.exp(z)), 0.0)
        wide.scatter_add_(1, at, d)
        d = wide[:, :K]
    if c["accumulate"]:
        s["grad"].copy_((s["grad"].view(-1, K).float() + d).view(s["grad"].shape))
        return s["grad"]
    return d.to(s["logits"].dtype).view(s["logits"].shape)


def _to_8bit(t, kind, top, least):
    """Codes and a factor per block of 32-bit values."""
    b = t.view(-1, BLOCK)
    high = b.abs().amax(-1, keepdim=True)
    y = b * torch.where(high > 0.0, top / high, 0.0)
    if least:
        y = torch.where(b > 0.0, y.clamp(min=least), y)
    return y.to(kind).view(-1), (high / top).view(-1)


def _adamw(s):
    c, r = s["case"], s["rate"]
    b1, b2 = r["betas"]
    g = s["g"].float()
    m, v = s["m"], s["v"]
    if c["bits"] == 8:
        m = (m.float().view(-1, BLOCK) * s["sm"][:, None]).view(-1)
        v = (v.float().view(-1, BLOCK) * s["sv"][:, None]).view(-1)
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    p = (s["p"] if s["master"] is None else s["master"]).float()
    step = m / (torch.sqrt(v) * (1.0 - b2 ** r["step"]) ** -0.5 + r["eps"])
    p = p * (1.0 - r["lr"] * r["weight_decay"]) - step * (r["lr"] / (1.0 - b1 ** r["step"]))
    if s["master"] is not None:
        s["master"].copy_(p)
    s["p"].copy_(p)
    if c["bits"] == 8:
        m, sm = _to_8bit(m, torch.float8_e4m3fn, 256.0, 0.0)
        v, sv = _to_8bit(v, torch.float8_e5m2, 32768.0, 2.0 ** -16)
        s["sm"].copy_(sm)
        s["sv"].copy_(sv)
    s["m"].copy_(m)
    s["v"].copy_(v)
    return _outputs(s)


def _outputs(s):
    return {k: s[k] for k in ("p", "master", "m", "v", "sm", "sv") if s[k] is not None}


# ---- the least a pass moves and computes ---------------------------------------------------------------------------------

def work(case):
    if case["op"] == "adamw":
        n, p = case["total"], BYTES[case["type"]]
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        weights = p + 8 if case["master"] else 2 * p
        return {"bytes": n * (weights + BYTES[case["grad"]] + state), "flops": 15 * n}
    B, N, K, S, e = case["B"], case["N"], case["K"], case["S"], BYTES[case["type"]]
    live = N - int(case["pad"] * N)
    if case["op"] == "route":
        return {"bytes": B * (live * K * e + N * S * 12 + (N if case["pad"] else 0)) + (4 * K if case["bias"] else 0),
                "flops": 5 * B * live * K}
    dense = case["score"] == "softmax" and not case["renorm"]
    if case["accumulate"]:
        out = 2 * live * K if dense else 2 * live * S
    else:
        out = N * K
    return {"bytes": B * (N * S * (8 if dense else 12) + out * e + (live * K * e if dense else 0)),
            "flops": 6 * B * live * (K if dense else S)}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_grad": _exact_route_grad, "adamw": _exact_adamw}[case["op"]](case, s)


def _exact_route(case, s):
    K, S, G = case["K"], case["S"], case["G"]
    x = s["logits"].reshape(-1, K).double()
    score = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    rank = x.clone()
    if s["bias"] is not None or (G > 1 and case["best"] == 2 and K > G):
        rank = score + (s["bias"].double() if s["bias"] is not None else 0.0)
        rank[x == -math.inf] = -math.inf
    if G > 1:
        rank = rank.reshape(-1, G, K // G)
        top = torch.topk(rank, min(case["best"], K // G), -1).values
        worth = torch.nan_to_num(top, neginf=0.0).sum(-1).masked_fill(top[..., 0] == -math.inf, -math.inf)
        # a group stays if fewer than `keep` are better, or as good and in front of it
        first = torch.arange(G, device="cuda")
        better = (worth[:, None, :] > worth[:, :, None]) | (
            (worth[:, None, :] == worth[:, :, None]) & (first[None, None, :] < first[None, :, None]))
        rank = rank.masked_fill((better.sum(-1) >= case["keep"])[..., None], -math.inf).reshape(-1, K)
    ids = torch.argsort(-rank, dim=-1, stable=True)[:, :S]
    out = rank.gather(1, ids) == -math.inf
    if s["valid"] is not None:
        out |= ~s["valid"].reshape(-1, 1)
    w = score.gather(1, ids).masked_fill(out, 0.0)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    shape = (*s["logits"].shape[:-1], S)
    return {"ids": ids.masked_fill(out, -1).reshape(shape), "weights": (w * case["scale"]).reshape(shape),
            "chosen": x.gather(1, ids).masked_fill(out, -math.inf).reshape(shape)}


def _exact_route_grad(case, s):
    K, S = case["K"], case["S"]
    x = s["logits"].reshape(-1, K).double()
    ids = s["ids"].reshape(-1, S).long()
    one_hot = torch.zeros((ids.shape[0], K + 1), dtype=torch.float64, device="cuda")
    have = torch.zeros_like(one_hot)
    at = ids.masked_fill(ids < 0, K)
    one_hot.scatter_add_(1, at, s["dweights"].reshape(-1, S).double())
    have.scatter_(1, at, 1.0)
    dw, have = one_hot[:, :K] * case["scale"], have[:, :K]
    if case["score"] == "softmax":
        if case["renorm"]:  # a softmax over the selected choices
            x = x.masked_fill(have == 0, -math.inf)
            x = x.masked_fill((have.sum(-1) == 0)[:, None], 0.0)
        p = torch.where((have.sum(-1) > 0)[:, None], torch.softmax(x, -1), 0.0)
        d = p * (dw - (p * dw).sum(-1, keepdim=True))
    else:
        f = torch.sigmoid(x) * have
        if case["renorm"]:
            total = f.sum(-1, keepdim=True).clamp(min=1e-300)
            dw = (dw - (f * dw).sum(-1, keepdim=True) / total) / total
        d = f * torch.sigmoid(-x) * dw
    d = d.masked_fill(have == 0, 0.0) if case["score"] == "sigmoid" or case["renorm"] else d
    d = d.reshape(s["logits"].shape)
    return d + s["grad"].double() if case["accumulate"] else d


def _exact_adamw(case, s):
    r = s["rate"]
    b1, b2 = r["betas"]
    g = s["g"].double()
    # the rates as 32-bit values, as the step holds them
    f = lambda x: float(torch.tensor(x, dtype=torch.float32))  # noqa: E731
    held = lambda code, factor: (code.double().view(-1, BLOCK) * factor.double()[:, None]).view(-1)  # noqa: E731
    m = s["m"].double() if case["bits"] == 32 else held(s["m"], s["sm"])
    v = s["v"].double() if case["bits"] == 32 else held(s["v"], s["sv"])
    m = f(b1) * m + f(1.0 - b1) * g
    v = f(b2) * v + f(1.0 - b2) * g.square()
    p = (s["p"] if s["master"] is None else s["master"]).double()
    p = p * (1.0 - r["lr"] * r["weight_decay"]) - r["lr"] / (1.0 - b1 ** r["step"]) * m / (
        torch.sqrt(v / (1.0 - b2 ** r["step"])) + r["eps"])
    out = {"p": p, "m": m, "v": v}
    if s["master"] is not None:
        out["master"] = p
    if case["bits"] == 8:
        for k, top in (("m", 256.0), ("v", 32768.0)):
            b = out[k].view(-1, BLOCK)
            high = b.abs().amax(-1, keepdim=True)
            out["s" + k] = (high / top).view(-1)
            out[k] = torch.where(high > 0.0, b / high * top, 0.0).view(-1)
    return out
