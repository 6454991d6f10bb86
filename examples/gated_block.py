"""A gated feed-forward block, as in LLaMA: trained over a tensor-parallel group,
with the group's ranks run in turn on one GPU, and served in 8 bits.

    python examples/gated_block.py [--tokens 2048 --hidden 1024 --ffn 2048 ...]

Training, per rank (sequence parallelism: a rank holds tokens / world rows):
RMS norm with the residual's addition -> all-gather + gate|up matmul -> gated
activation -> down matmul + reduce-scatter, and the backward pass down to the
rows, the norm's gamma and the two weights' shards.  With one rank the
projections and the activation are one call (gated_ffn) instead.

Serving: the weights once in 8 bits, then norm -> product -> activation ->
product with 8-bit operands, for a prompt or for single tokens; the ranks'
partial outputs are added.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import tensor_gemm_collective_amd as tgc  # noqa: E402


def make_params(world, hidden, ffn, seed=0, device="cuda", dtype=torch.bfloat16):
    """gamma, and by rank the gate|up shard (hidden x 2 ffn/world) and the down shard (ffn/world x hidden)."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, sigma):
        return (torch.randn(shape, generator=g) * sigma).to(dtype).to(device)

    f = ffn // world
    return {"gamma": normal(hidden, sigma=0.1) + 1.0,
            "w": [normal(hidden, 2 * f, sigma=hidden ** -0.5) for _ in range(world)],
            "down": [normal(f, hidden, sigma=ffn ** -0.5) for _ in range(world)]}


def forward(p, rows, residual, act):
    """rows[r], residual[r]: rank r's tokens / world rows of the layer's input and of the
    residual stream.  Returns the ranks' outputs and what the backward pass needs."""
    world = len(rows)
    normed, saved = [], []
    for r in range(world):
        y, rstd, total = tgc.rms_norm(rows[r], p["gamma"], residual=residual[r])
        normed.append(y)
        saved.append({"rstd": rstd, "sum": total})
    partials = []
    for r in range(world):
        if world == 1:
            h, both = tgc.gated_ffn(normed[0], p["w"][0], act=act, save=True)
            gathered = normed[0]
        else:
            both, gathered = tgc.allgather_matmul(normed[r], normed, p["w"][r], r, split=1, v2=True)
            h = tgc.gated_act(both, act=act)
        saved[r] |= {"both": both, "x": gathered, "h": h}
        # what this rank hands to the others (their sums follow below)
        zeros = [torch.zeros(h.shape[0], rows[0].shape[1], dtype=h.dtype, device=h.device)] * world
        partials.append(tgc.matmul_reduce_scatter(h, p["down"][r], zeros, r, split=1)[1])
    outs = []
    for r in range(world):
        y, _ = tgc.matmul_reduce_scatter(saved[r]["h"], p["down"][r], partials, r, split=1)
        outs.append(y)
    return outs, saved


def backward(p, douts, dsum, act, saved):
    """Gradients of sum <out, dout> + <sum, dsum> by the ranks' rows (the same by their
    residual), gamma and the weights' shards."""
    world = len(douts)
    grads = {"gamma": 0.0, "w": [], "down": [], "rows": []}
    partials = []
    for r in range(world):
        s = saved[r]
        # the reduce-scatter's gradient is an all-gather, and the all-gather's a reduce-scatter
        dh, dy = tgc.allgather_matmul(douts[r], douts, p["down"][r], r, split=1, v2=True, trans_w=True)
        grads["down"].append(tgc.weight_grad(s["h"], dy))
        if world == 1:
            dx, dw = tgc.gated_ffn_backward(dh, s["x"], p["w"][0], s["both"], act=act)
            grads["w"].append(dw)
            partials.append(dx)
            continue
        dboth = tgc.gated_act_backward(dh, s["both"], act=act)
        grads["w"].append(tgc.weight_grad(s["x"], dboth))
        s["dboth"] = dboth
        zeros = [torch.zeros_like(s["x"])] * world
        partials.append(tgc.matmul_reduce_scatter(dboth, p["w"][r], zeros, r, split=1, trans_w=True)[1])
    for r in range(world):
        s = saved[r]
        dy = partials[0] if world == 1 else tgc.matmul_reduce_scatter(s["dboth"], p["w"][r], partials, r, split=1,
                                                                      trans_w=True)[0]
        dx, dgamma = tgc.rms_norm_backward(dy, s["sum"], p["gamma"], s["rstd"], dsum=dsum[r])
        grads["rows"].append(dx)
        grads["gamma"] = grads["gamma"] + dgamma.float()
    return grads


def weights_fp8(p, rank=0):
    """A rank's weights in 8 bits, as rows of the products' inputs: gate|up, down."""
    return {name: tgc.quantize_fp8(p[key][rank].t().contiguous(), block_rows=128)
            for name, key in (("w", "w"), ("down", "down"))}


def serve(p, w8, x, residual, act):
    """One rank's part of the block in 8 bits: (its partial output, the residual stream)."""
    q, scales, _, total = tgc.rms_norm_fp8(x, p["gamma"], residual=residual)
    both = tgc.matmul_fp8(q, scales, *w8["w"], dtype=x.dtype)
    q, scales = tgc.gated_act_fp8(both, act=act)
    return tgc.matmul_fp8(q, scales, *w8["down"], dtype=x.dtype), total


def serve_group(p, w8, x, residual, act):
    """The block in 8 bits over the ranks, whose weights w8 lists: (output, residual stream).
    What an all-reduce does over a group of GPUs, the partial outputs' sum, is taken here
    in binary32 and rounded once."""
    parts = [serve(p, w, x, residual, act) for w in w8]
    out = parts[0][0].float()
    for part, _ in parts[1:]:
        out = out + part.float()
    return out.to(x.dtype), parts[0][1]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("world", 2), ("tokens", 2048), ("hidden", 1024), ("ffn", 2048), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--act", choices=("silu", "gelu"), default="silu")
    a = ap.parse_args()
    p = make_params(a.world, a.hidden, a.ffn)
    g = torch.Generator().manual_seed(1)
    share = a.tokens // a.world

    def rows():
        return [torch.randn(share, a.hidden, generator=g).bfloat16().cuda() for _ in range(a.world)]

    x, residual, douts, dsum = rows(), rows(), rows(), rows()
    w8 = [weights_fp8(p, r) for r in range(a.world)]
    prompt, token = (torch.randn(n, a.hidden, generator=g).bfloat16().cuda() for n in (a.tokens, 1))

    def timed(what, f):
        f()
        torch.cuda.synchronize()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            out = f()
        end.record()
        torch.cuda.synchronize()
        print(f"{what}: {start.elapsed_time(end) / a.steps * 1e3:.1f} us")
        return out

    def step():
        outs, saved = forward(p, x, residual, a.act)
        return outs, backward(p, douts, dsum, a.act, saved)

    outs, grads = timed(f"step of {a.world} ranks x {share} tokens, hidden {a.hidden}, ffn {a.ffn}", step)
    for what, t in ((f"{a.tokens} tokens", prompt), ("1 token", token)):
        timed(f"8 bits, {what}, one rank's part", lambda: serve(p, w8[0], t, t, a.act))
        timed(f"8 bits, {what}, {a.world} ranks in turn", lambda: serve_group(p, w8, t, t, a.act))
    print(f"|out| {float(torch.stack([o.float().norm() for o in outs]).norm()):.1f}, "
          f"|d rows| {float(torch.stack([d.float().norm() for d in grads['rows']]).norm()):.1f}")


if __name__ == "__main__":
    main()
