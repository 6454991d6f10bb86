"""Cases and plain forms of the operators around the fused matmul/collective ops.

One tensor- or expert-parallel rank's share of a training step, next to the
matmuls: the embedding lookup in front of the layers, the layer norm in front
of every column-parallel matmul, and in a MoE layer the router (selection,
per-expert counts, balance loss) with the row moves into and out of the
experts' all-to-all.

A case is a dict whose "op" names the operator; `prepare` makes what a
training program holds before the call, `run` makes one pass.  With `own`
false `run` computes the plain form in elementary torch operations; with `own`
true it calls the library.  `exact` is the operators' definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
COEF = 0.01
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token's final norm at the widest hidden size, as in decoding
        {"name": "ln_token", "op": "layer_norm", "rows": 1, "n": 14336, "dtype": "bf16", "residual": False},
        # a rank's sequence shard (4096 / 8 rows) with the residual sum in front of the all-gather matmul
        {"name": "ln_shard", "op": "layer_norm", "rows": 512, "n": 8192, "dtype": "bf16", "residual": True},
        # the norm's backward without sequence parallelism, residual gradient joined in
        {"name": "ln_backward", "op": "layer_norm_backward", "rows": 2048, "n": 14336, "dtype": "bf16",
         "residual": True},
        # a rank's vocabulary shard, most of the ids belonging to other ranks
        {"name": "embed_shard", "op": "embedding", "tokens": 4096, "vocab": 4000, "world": 8, "n": 8192,
         "dtype": "bf16"},
        # a small odd-sized table in 32 bits
        {"name": "embed_grad_odd", "op": "embedding_grad", "tokens": 1001, "vocab": 1999, "world": 1, "n": 515,
         "dtype": "f32"},
        # the whole table's gradient of a long batch, ids as skewed as words are
        {"name": "embed_grad", "op": "embedding_grad", "tokens": 32768, "vocab": 32000, "world": 1, "n": 4096,
         "dtype": "bf16"},
        # a short ragged batch routed over 8 ranks in 4 pieces, padding masked
        {"name": "router_small", "op": "moe_router", "tokens": 300, "experts": 16, "topk": 2, "pieces": 4, "world": 8,
         "dtype": "f16", "masked": True, "renormalize": True},
        # a long batch over as many experts as the all-to-all takes
        {"name": "router_large", "op": "moe_router", "tokens": 65536, "experts": 128, "topk": 8, "pieces": 2,
         "world": 8, "dtype": "bf16", "masked": False, "renormalize": True},
        # the router's gradient from the gates' and the balance loss's
        {"name": "router_backward", "op": "moe_router_backward", "tokens": 65536, "experts": 64, "topk": 4,
         "pieces": 2, "world": 8, "dtype": "f32", "masked": True, "renormalize": False},
        # rows of a short ragged batch into their send order
        {"name": "permute_small", "op": "moe_permute", "tokens": 300, "n": 130, "experts": 16, "topk": 2, "pieces": 4,
         "world": 8, "dtype": "f16"},
        # the experts' rows summed by their gates: 8192 tokens of 12288, 4 experts, top 2
        {"name": "combine", "op": "moe_combine", "tokens": 8192, "n": 12288, "experts": 4, "topk": 2, "pieces": 2,
         "world": 2, "dtype": "bf16"},
        # and its backward pass
        {"name": "combine_backward", "op": "moe_combine_backward", "tokens": 8192, "n": 12288, "experts": 4, "topk": 2,
         "pieces": 2, "world": 2, "dtype": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi, odd=0.3):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return v | 1 if rng.random() < odd and v < hi else v

    op = rng.choice(["layer_norm", "layer_norm_backward", "embedding", "embedding_grad", "moe_router",
                     "moe_router_backward", "moe_permute", "moe_combine", "moe_combine_backward"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op.startswith("layer_norm"):
        n = spread(64, 14336)
        rows = spread(1, max(2, min(16384, 2048 * 14336 // n)))
        return {"op": op, "rows": rows, "n": n, "dtype": dtype, "residual": rng.random() < 0.5}
    if op.startswith("embedding"):
        world = rng.choice([1, 2, 8])
        n = spread(64, 8192)
        tokens = spread(1, max(2, min(32768, 32768 * 4096 // n)))
        vocab = spread(16, max(32, min(32000, 32000 * 4096 // n)))
        return {"op": op, "tokens": tokens, "vocab": vocab, "world": world, "n": n, "dtype": dtype}
    world = rng.choice([1, 2, 8])
    experts = world * rng.choice([1, 2, 3, 4, 5, 8, 16])
    topk = rng.randint(1, min(8, experts))
    case = {"op": op, "tokens": 0, "experts": experts, "topk": topk, "pieces": rng.choice([1, 2, 4, 8]), "world": world,
            "dtype": dtype}
    if op.startswith("moe_router"):
        case["tokens"] = spread(1, 65536)
        case["masked"] = rng.random() < 0.5
        case["renormalize"] = rng.random() < 0.5
        return case
    case["n"] = spread(64, 12288)
    rows = {"moe_permute": 1 + topk, "moe_combine": 1 + topk, "moe_combine_backward": 1 + 2 * topk}[op]
    case["tokens"] = spread(1, max(2, min(32768, 980_000_000 // (case["n"] * _size(case) * rows))))
    return case


# ------------------------------------------------------------------ inputs
def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def _normal(gen, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)


def _logits(case, gen):
    # the experts are not equally liked
    bias = 0.7 * torch.randn(case["experts"], generator=gen, device="cuda")
    raw = 1.3 * torch.randn(case["tokens"], case["experts"], generator=gen, device="cuda")
    return (raw + bias).to(DTYPES[case["dtype"]])


def _mask(case, gen):
    """The padding of a batch: about a tenth of the tokens, in runs of 16."""
    if not case["masked"]:
        return None
    runs = (case["tokens"] + 15) // 16
    keep = torch.rand(runs, generator=gen, device="cuda") >= 0.1
    return keep.repeat_interleave(16)[:case["tokens"]].to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    if op.startswith("layer_norm"):
        rows, n = case["rows"], case["n"]
        s["x"] = _normal(gen, (rows, n), dt, 1.5) + 0.25
        s["gamma"] = _normal(gen, (n,), dt, 0.1) + 1.0
        s["beta"] = _normal(gen, (n,), dt, 0.1)
        s["other"] = _normal(gen, (rows, n), dt) if case["residual"] else None
        if op == "layer_norm_backward":
            s["dy"] = _normal(gen, (rows, n), dt)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = (x - s["mean"][:, None]).square().mean(1).add(EPS).rsqrt()
    elif op.startswith("embedding"):
        tokens, vocab, n = case["tokens"], case["vocab"], case["n"]
        every = vocab * case["world"]
        # the frequency of an id falls with its rank; which id has which rank is shuffled
        rank = torch.rand(tokens, generator=gen, device="cuda", dtype=torch.float64)
        rank = torch.exp(rank * math.log(every)).long().clamp(1, every) - 1
        s["ids"] = torch.randperm(every, generator=gen, device="cuda")[rank]
        s["start"] = vocab * (case["world"] // 2)
        s["scale"] = math.sqrt(n)
        if op == "embedding":
            s["table"] = _normal(gen, (vocab, n), dt, 0.02)
        else:
            s["dy"] = _normal(gen, (tokens, n), dt, 0.1)
    elif op.startswith("moe_router"):
        s["logits"] = _logits(case, gen)
        s["mask"] = _mask(case, gen)
        if op == "moe_router_backward":
            r = _router(s)
            s["ids"], s["gates"], s["counts"], s["valid"] = r["ids"], r["gates"], r["counts"], r["valid"]
            s["dgates"] = _normal(gen, (case["tokens"], case["topk"]), torch.float32)
            s["dloss"] = torch.full((1,), 1.0 + 0.001 * (seed % 1000), device="cuda")
    else:
        tokens, n, k = case["tokens"], case["n"], case["topk"]
        logits = _logits(case, gen).float()
        chosen = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
        s["positions"] = _positions(chosen, s)
        if op == "moe_permute":
            s["x"] = _normal(gen, (tokens, n), dt)
        else:
            s["h"] = _normal(gen, (tokens * k, n), dt)
            s["gates"] = torch.softmax(torch.gather(logits, 1, chosen), 1).contiguous()
            if op == "moe_combine_backward":
                s["dy"] = _normal(gen, (tokens, n), dt)
    return s


# ------------------------------------------------------------------ plain forms
def _positions(ids, s):
    """The send row of every (token, choice): by destination rank, then piece of
    the sequence, then expert, then token; -1 where nothing was chosen."""
    tokens, experts, pieces = s["tokens"], s["experts"], s["pieces"]
    local = experts // s["world"]
    ends = torch.arange(1, pieces, device="cuda") * tokens // pieces
    piece = torch.bucketize(torch.arange(tokens, device="cuda"), ends, right=True)[:, None]
    key = ((ids // local) * pieces + piece) * local + ids % local
    key = torch.where(ids >= 0, key, experts * pieces).reshape(-1)
    order = torch.sort(key, stable=True)[1]
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    return torch.where(ids >= 0, pos.view_as(ids), -1).to(torch.int32)


def _softmax(s):
    """Logits in 32 bits, exp(logit - max), its row sums, and the rows that take part."""
    x = s["logits"].float()
    top = x.max(1, keepdim=True)[0]
    live = top != -math.inf
    if s["mask"] is not None:
        live = live & (s["mask"] != 0)[:, None]
    e = torch.where(live, torch.exp(x - top), 0.0)
    return x, e, e.sum(1, keepdim=True), live


def _router(s):
    tokens, experts, k, pieces = s["tokens"], s["experts"], s["topk"], s["pieces"]
    x, e, total, live = _softmax(s)
    p = torch.where(live, e / total, 0.0)
    value, ids = torch.sort(x, dim=1, descending=True, stable=True)
    ids = torch.where(live & (value[:, :k] != -math.inf), ids[:, :k], -1)
    chosen = torch.where(ids >= 0, torch.gather(e, 1, ids.clamp(min=0)), 0.0)
    under = chosen.sum(1, keepdim=True) if s["renormalize"] else total
    gates = torch.where(ids >= 0, chosen / under, 0.0)
    ends = torch.arange(1, pieces, device="cuda") * tokens // pieces
    piece = torch.bucketize(torch.arange(tokens, device="cuda"), ends, right=True)[:, None]
    slot = torch.where(ids >= 0, piece * experts + ids, pieces * experts).reshape(-1)
    counts = torch.zeros(pieces * experts + 1, dtype=torch.int64, device="cuda")
    counts = counts.index_add_(0, slot, torch.ones_like(slot))[:-1].view(pieces, experts)
    valid = live.sum().view(1)
    prob_sums = p.sum(0)
    n = valid.clamp(min=1).float()
    loss = COEF * experts / k * (counts.sum(0).float() / n * (prob_sums / n)).sum().view(1)
    return {"ids": ids.to(torch.int32), "gates": gates, "positions": _positions(ids, s), "counts": counts,
            "prob_sums": prob_sums, "loss": loss, "valid": valid}


def _router_backward(s):
    k, experts = s["topk"], s["experts"]
    _, e, total, live = _softmax(s)
    p = torch.where(live, e / total, 0.0)
    n = s["valid"].clamp(min=1).float()
    a = s["dloss"] * COEF * experts / k * s["counts"].sum(0).float() / (n * n)
    out = p * (a - (p * a).sum(1, keepdim=True))
    ids = s["ids"].long()
    g = s["gates"]
    dg = torch.where(ids >= 0, s["dgates"], 0.0)
    at = ids.clamp(min=0)
    inner = (g * dg).sum(1, keepdim=True)
    if s["renormalize"]:
        out = out.scatter_add(1, at, g * (dg - inner))
    else:
        out = (out - p * inner).scatter_add(1, at, g * dg)
    return torch.where(live, out, 0.0).to(s["logits"].dtype)


def _plain(s):
    op = s["op"]
    if op == "layer_norm":
        x = s["x"]
        if s["residual"]:
            x = (x.float() + s["other"].float()).to(x.dtype)
        h = x.float()
        mean = h.mean(1)
        d = h - mean[:, None]
        rstd = 1.0 / torch.sqrt(d.square().mean(1) + EPS)
        y = (d * rstd[:, None] * s["gamma"].float() + s["beta"].float()).to(x.dtype)
        return {"y": y, "mean": mean, "rstd": rstd, "sum": x if s["residual"] else None}
    if op == "layer_norm_backward":
        dy = s["dy"].float()
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["gamma"].float()
        dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        if s["residual"]:
            dx = dx + s["other"].float()
        return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0).to(s["gamma"].dtype),
                "dbeta": dy.sum(0).to(s["gamma"].dtype)}
    if op.startswith("embedding"):
        vocab = s["vocab"]
        local = s["ids"] - s["start"]
        mine = (local >= 0) & (local < vocab)
    if op == "embedding":
        rows = s["table"][torch.where(mine, local, 0)].float() * s["scale"]
        return torch.where(mine[:, None], rows, 0.0).to(s["table"].dtype)
    if op == "embedding_grad":
        total = torch.zeros(vocab + 1, s["n"], device="cuda")
        total.index_add_(0, torch.where(mine, local, vocab), s["dy"].float())
        return (total[:vocab] * s["scale"]).to(s["dy"].dtype)
    if op == "moe_router":
        return _router(s)
    if op == "moe_router_backward":
        return _router_backward(s)
    pos = s["positions"].long()
    if op == "moe_permute":
        x = s["x"]
        out = torch.empty(pos.numel(), s["n"], dtype=x.dtype, device="cuda")
        out[pos.reshape(-1)] = x[:, None, :].expand(-1, s["topk"], -1).reshape(pos.numel(), s["n"])
        return out
    h = s["h"][pos].float()
    if op == "moe_combine":
        return (s["gates"][:, :, None] * h).sum(1).to(s["h"].dtype)
    dy = s["dy"].float()[:, None, :]
    dh = torch.empty_like(s["h"])
    dh[pos.reshape(-1)] = (s["gates"][:, :, None] * dy).to(dh.dtype).view(pos.numel(), s["n"])
    return {"dh": dh, "dgates": (dy * h).sum(2)}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import tensor_gemm_collective_amd as tgc
    op = s["op"]
    if op == "layer_norm":
        got = tgc.layer_norm(s["x"], s["gamma"], s["beta"], residual=s["other"], eps=EPS)
        return {"y": got[0], "mean": got[1], "rstd": got[2], "sum": got[3] if s["residual"] else None}
    if op == "layer_norm_backward":
        dx, dgamma, dbeta = tgc.layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"],
                                                    dsum=s["other"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "embedding":
        return tgc.embedding(s["ids"], s["table"], start=s["start"], scale=s["scale"])
    if op == "embedding_grad":
        return tgc.embedding_grad(s["ids"], s["dy"], s["vocab"], start=s["start"], scale=s["scale"])
    if op == "moe_router":
        r = tgc.moe_router(s["logits"], s["topk"], pieces=s["pieces"], world=s["world"], coef=COEF,
                           renormalize=s["renormalize"], mask=s["mask"])
        return {"ids": r.ids, "gates": r.gates, "positions": r.positions, "counts": r.counts,
                "prob_sums": r.prob_sums, "loss": r.loss, "valid": r.valid}
    if op == "moe_router_backward":
        return tgc.moe_router_backward(s["logits"], s["ids"], s["gates"], s["counts"], s["valid"], s["dgates"],
                                       s["dloss"], coef=COEF, renormalize=s["renormalize"], mask=s["mask"])
    if op == "moe_permute":
        return tgc.moe_permute(s["x"], s["positions"])
    if op == "moe_combine":
        return tgc.moe_combine(s["h"], s["positions"], s["gates"])
    dh, dgates = tgc.moe_combine_backward(s["dy"], s["h"], s["positions"], s["gates"])
    return {"dh": dh, "dgates": dgates}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, es = case["op"], _size(case)
    if op.startswith("layer_norm"):
        rows, n = case["rows"], case["n"]
        if op == "layer_norm":
            return {"bytes": es * (rows * n * (4 if case["residual"] else 2) + 2 * n) + 8 * rows, "flops": 8 * rows * n}
        return {"bytes": es * (rows * n * (4 if case["residual"] else 3) + 3 * n) + 8 * rows, "flops": 16 * rows * n}
    if op.startswith("embedding"):
        # rows of other ranks' ids are not read; about 1 / world of the tokens are this rank's, and with repeated ids
        # the lookup reads at most each table row once
        tokens, n = case["tokens"], case["n"]
        mine = tokens / case["world"]
        if op == "embedding":
            return {"bytes": es * n * (tokens + min(mine, case["vocab"])) + 8 * tokens, "flops": mine * n}
        return {"bytes": es * n * (mine + case["vocab"]) + 8 * tokens, "flops": mine * n + case["vocab"] * n}
    tokens, k, experts = case["tokens"], case["topk"], case["experts"]
    if op.startswith("moe_router"):
        mask = tokens if case["masked"] else 0
        if op == "moe_router":
            return {"bytes": tokens * (es * experts + 12 * k) + mask + 8 * case["pieces"] * experts + 4 * experts + 12,
                    "flops": 6 * tokens * experts}
        return {"bytes": tokens * (2 * es * experts + 12 * k) + mask + 8 * case["pieces"] * experts + 12,
                "flops": 10 * tokens * experts}
    n = case["n"]
    if op == "moe_permute":
        return {"bytes": es * tokens * n * (1 + k) + 4 * tokens * k, "flops": 0}
    if op == "moe_combine":
        return {"bytes": es * tokens * n * (1 + k) + 8 * tokens * k, "flops": 2 * tokens * n * k}
    return {"bytes": es * tokens * n * (1 + 2 * k) + 12 * tokens * k, "flops": 3 * tokens * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_router(s):
    """Token by token: softmax, the chosen experts' gates, and the loss as the
    mean share of the choices times the mean probability."""
    x = s["logits"].double()
    keep = ~torch.isneginf(x).all(1)
    if s["mask"] is not None:
        keep &= s["mask"].bool()
    p = torch.zeros_like(x)
    p[keep] = torch.softmax(x[keep], 1)
    return p, keep


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "layer_norm":
        h = s["x"].double()
        if s["residual"]:
            h = (s["x"].double() + s["other"].double()).to(s["x"].dtype).double()
        mean = h.sum(1) / s["n"]
        var = (h * h).sum(1) / s["n"] - mean * mean
        rstd = (var + EPS) ** -0.5
        y = (h * rstd[:, None] - (mean * rstd)[:, None]) * s["gamma"].double() + s["beta"].double()
        return {"y": y, "mean": mean, "rstd": rstd, "sum": h if s["residual"] else None}
    if op == "layer_norm_backward":
        # the Jacobian of (x - mean) * rstd applied to dy * gamma: two projections taken off
        dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
        c = s["x"].double() - s["mean"].double()[:, None]
        v = dy * s["gamma"].double() * rstd
        dx = v - v.sum(1, keepdim=True) / s["n"] - c * ((v * c).sum(1, keepdim=True) * rstd * rstd / s["n"])
        if s["residual"]:
            dx += s["other"].double()
        return {"dx": dx, "dgamma": torch.mv(c.t() * dy.t(), rstd[:, 0]),
                "dbeta": torch.mv(dy.t(), torch.ones_like(rstd[:, 0]))}
    if op == "embedding":
        y = torch.zeros(s["tokens"], s["n"], dtype=torch.float64, device="cuda")
        at = ((s["ids"] >= s["start"]) & (s["ids"] < s["start"] + s["vocab"])).nonzero()[:, 0]
        y[at] = s["table"].double()[s["ids"][at] - s["start"]] * s["scale"]
        return y
    if op == "embedding_grad":
        g = torch.zeros(s["vocab"], s["n"], dtype=torch.float64, device="cuda")
        at = ((s["ids"] >= s["start"]) & (s["ids"] < s["start"] + s["vocab"])).nonzero()[:, 0]
        if at.numel():
            g.index_put_((s["ids"][at] - s["start"],), s["scale"] * s["dy"][at].double(), accumulate=True)
        return g
    if op == "moe_router":
        p, keep = _exact_router(s)
        x = s["logits"].double()
        at = torch.argsort(-x, dim=1, stable=True)[:, :s["topk"]]
        at = at.masked_fill(~keep[:, None] | torch.isneginf(x.gather(1, at)), -1)
        g = torch.where(at >= 0, p.gather(1, at.clamp(min=0)), 0.0)
        if s["renormalize"]:
            g = g / g.sum(1, keepdim=True).clamp(min=1e-300)
        n = max(1, int(keep.sum()))
        share = torch.bincount(at[at >= 0], minlength=s["experts"]).double() / (n * s["topk"])
        loss = COEF * s["experts"] * torch.dot(share, p.sum(0) / n).view(1)
        return {"ids": None, "gates": g, "positions": None, "counts": None, "prob_sums": p.sum(0), "loss": loss,
                "valid": None}
    if op == "moe_router_backward":
        p, keep = _exact_router(s)
        at = s["ids"].long()
        n = max(1, int(keep.sum()))
        share = torch.bincount(at[at >= 0], minlength=s["experts"]).double() / (n * s["topk"])
        dp = (s["dloss"].double() * COEF * s["experts"] / n * share).repeat(s["tokens"], 1)
        g = p.gather(1, at.clamp(min=0)) * (at >= 0)
        dg = s["dgates"].double() * (at >= 0)
        if s["renormalize"]:
            total = g.sum(1, keepdim=True).clamp(min=1e-300)
            dg = (dg - (dg * g).sum(1, keepdim=True) / total) / total * (at >= 0)
        dp.scatter_add_(1, at.clamp(min=0), dg)
        return p * dp - p * (p * dp).sum(1, keepdim=True)
    pos = s["positions"].long()
    token = torch.arange(s["tokens"], device="cuda").repeat_interleave(s["topk"])
    back = torch.empty_like(token)
    back[pos.reshape(-1)] = torch.arange(pos.numel(), device="cuda")
    if op == "moe_permute":
        return s["x"][token[back]].double()
    if op == "moe_combine":
        y = torch.zeros(s["tokens"], s["n"], dtype=torch.float64, device="cuda")
        return y.index_add_(0, token[back], s["h"].double() * s["gates"].reshape(-1)[back].double()[:, None])
    dy = s["dy"].double()[token[back]]
    dgates = torch.empty(pos.numel(), dtype=torch.float64, device="cuda")
    dgates[back] = (dy * s["h"].double()).sum(1)
    return {"dh": dy * s["gates"].reshape(-1)[back].double()[:, None], "dgates": dgates.view(pos.shape)}
