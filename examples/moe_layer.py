"""One step of a MoE layer over an expert-parallel group, forward and backward,
with the group's ranks run in turn on one GPU.

    python examples/moe_layer.py [--tokens 2048 --hidden 1024 --ffn 2048 ...]

Per rank: embedding lookup (the vocabulary in shards, one a rank) -> layer norm
-> router -> rows into their send order -> dispatch all-to-all + the experts'
first matmul -> GELU -> the second matmul + combine all-to-all -> the rows'
gate-weighted sum, plus the residual.  The balance loss is added to the step's
loss.  Backward: every operator's gradient down to the embedding shards, the
norm's gamma and beta and the router's weight (the expert weights' gradients
are left out: weight_grad takes them group by group).

The router's product (hidden x experts) and the activation are torch's.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_gemm_collective_amd as tgc  # noqa: E402


def make_params(world, vocab, hidden, ffn, experts, seed=0, device="cuda", dtype=torch.bfloat16):
    """The layer's parameters: vocabulary shards and expert weights by rank."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, sigma):
        return (torch.randn(shape, generator=g) * sigma).to(dtype).to(device)

    local = experts // world
    return {
        "tables": [normal(vocab // world, hidden, sigma=1.0) for _ in range(world)],
        "gamma": normal(hidden, sigma=0.1) + 1.0,
        "beta": normal(hidden, sigma=0.1),
        "router": normal(hidden, experts, sigma=hidden ** -0.5),
        "w1": [normal(local, hidden, ffn, sigma=hidden ** -0.5) for _ in range(world)],
        "w2": [normal(local, ffn, hidden, sigma=ffn ** -0.5) for _ in range(world)],
    }


def _counts_to(rank, routings, local):
    """counts[piece][source][expert] of the rows that come to `rank`."""
    mine = torch.stack([r.counts[:, rank * local:(rank + 1) * local] for r in routings], dim=1)
    return mine.cpu().numpy()   # the pair takes its counts from the host


def _send_blocks(counts):
    """Where each destination's rows begin in a rank's send order (destination first)."""
    rows = [int(c.sum()) for c in counts]
    return [sum(rows[:d]) for d in range(len(rows) + 1)]


def forward(p, ids, masks, topk, pieces, coef):
    """ids[r], masks[r]: rank r's tokens.  Returns the ranks' outputs, their
    balance losses and what the backward pass needs."""
    world, experts = len(ids), p["router"].shape[1]
    local, vocab = experts // world, p["tables"][0].shape[0]
    saved, routings, sends = [], [], []
    for r in range(world):
        # each rank looks up its shard's ids; the sum over ranks is the whole lookup (an all-reduce)
        h = sum(tgc.embedding(ids[r], t, start=s * vocab) for s, t in enumerate(p["tables"]))
        y, mean, rstd = tgc.layer_norm(h, p["gamma"], p["beta"])
        logits = y.float() @ p["router"].float()
        route = tgc.moe_router(logits, topk, pieces=pieces, world=world, coef=coef, mask=masks[r])
        rows = tgc.moe_permute(y, route.positions)
        saved.append({"h": h, "y": y, "mean": mean, "rstd": rstd, "logits": logits})
        routings.append(route)
        sends.append(rows)
    counts = [_counts_to(r, routings, local) for r in range(world)]
    begin = [_send_blocks([c[:, r] for c in counts]) for r in range(world)]   # of source r, by destination

    def block(t, source, dest):
        return t[begin[source][dest]:begin[source][dest + 1]]

    returned = [torch.empty_like(s) for s in sends]
    for r in range(world):
        src = [block(sends[s], s, r) for s in range(world)]
        z, recv = tgc.alltoall_grouped_matmul(src[r], src, counts[r], p["w1"][r], r)
        act = torch.nn.functional.gelu(z.float(), approximate="tanh").to(z.dtype)
        back = [block(returned[s], s, r) for s in range(world)]
        tgc.grouped_matmul_alltoall(act, p["w2"][r], counts[r], r, y_own=back[r], peer_out=back)
        saved[r]["z"] = z
    outs = []
    for r in range(world):
        out = tgc.moe_combine(returned[r], routings[r].positions, routings[r].gates)
        outs.append(out + saved[r]["h"])
        saved[r]["rows"] = returned[r]
    return outs, [r.loss for r in routings], (saved, routings, counts, block)


def backward(p, ids, masks, douts, coef, state):
    """Gradients by the embedding shards, gamma, beta and the router's weight of
    sum <out, dout> + the sum of the balance losses."""
    saved, routings, counts, block = state
    world, vocab = len(ids), p["tables"][0].shape[0]
    one = torch.ones(1, device=douts[0].device)
    grads = {"tables": [torch.zeros(t.shape, device=t.device) for t in p["tables"]],
             "gamma": 0.0, "beta": 0.0, "router": 0.0}
    dgates, dsends, dreturned = [], [], []
    for r in range(world):
        drows, dg = tgc.moe_combine_backward(douts[r], saved[r]["rows"], routings[r].positions, routings[r].gates)
        dgates.append(dg)
        dreturned.append(drows)
        dsends.append(torch.empty_like(drows))
    for r in range(world):
        # the combine's gradient is a dispatch, and the dispatch's a combine, with the weights transposed
        src = [block(dreturned[s], s, r) for s in range(world)]
        dact, _ = tgc.alltoall_grouped_matmul(src[r], src, counts[r], p["w2"][r].transpose(1, 2).contiguous(), r)
        z = saved[r]["z"].float()
        inner = 0.7978845608028654 * (z + 0.044715 * z ** 3)
        t = torch.tanh(inner)
        slope = 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * z * z)
        dz = (dact.float() * slope).to(dact.dtype)
        back = [block(dsends[s], s, r) for s in range(world)]
        tgc.grouped_matmul_alltoall(dz, p["w1"][r].transpose(1, 2).contiguous(), counts[r], r, y_own=back[r],
                                    peer_out=back)
    for r in range(world):
        s, route = saved[r], routings[r]
        dy = tgc.moe_combine(dsends[r], route.positions)      # the gradient of the permutation
        dlogits = tgc.moe_router_backward(s["logits"], route.ids, route.gates, route.counts, route.valid, dgates[r],
                                          one, coef=coef, mask=masks[r])
        grads["router"] = grads["router"] + s["y"].float().t() @ dlogits
        dy = dy + (dlogits @ p["router"].float().t()).to(dy.dtype)
        dh, dgamma, dbeta = tgc.layer_norm_backward(dy, s["h"], p["gamma"], s["mean"], s["rstd"], dsum=douts[r])
        grads["gamma"] = grads["gamma"] + dgamma.float()
        grads["beta"] = grads["beta"] + dbeta.float()
        for i, g in enumerate(grads["tables"]):
            tgc.embedding_grad(ids[r], dh, vocab, start=i * vocab, grad=g, accumulate=True)
    return grads


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("world", 2), ("tokens", 2048), ("vocab", 8192), ("hidden", 1024), ("ffn", 2048),
                        ("experts", 8), ("topk", 2), ("pieces", 2), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    coef = 0.01
    p = make_params(a.world, a.vocab, a.hidden, a.ffn, a.experts)
    g = torch.Generator().manual_seed(1)
    ids = [torch.randint(0, a.vocab, (a.tokens,), generator=g).cuda() for _ in range(a.world)]
    masks = [(torch.rand(a.tokens, generator=g) > 0.05).cuda() for _ in range(a.world)]
    douts = [torch.randn(a.tokens, a.hidden, generator=g).bfloat16().cuda() for _ in range(a.world)]
    for step in range(a.steps + 1):
        if step == 1:
            torch.cuda.synchronize()
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
        outs, losses, state = forward(p, ids, masks, a.topk, a.pieces, coef)
        grads = backward(p, ids, masks, douts, coef, state)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.world} ranks x {a.tokens} tokens, hidden {a.hidden}, ffn {a.ffn}, {a.experts} experts, top {a.topk}: "
          f"{start.elapsed_time(end) / a.steps:.3f} ms a step; balance losses "
          f"{', '.join('%.4f' % float(v) for v in losses)}; |out| {float(outs[0].float().norm()):.1f}, "
          f"|d embedding| {float(torch.stack([t.norm() for t in grads['tables']]).norm()):.1f}")


if __name__ == "__main__":
    main()
