"""examples/moe_layer.py, a MoE layer's step made of the library's operators,
against the same layer in float64 with torch's autograd on the CPU.

Tolerance, normwise: every value that the layer keeps in bf16 carries a rounding
of at most 2^-8 of itself; at most 12 such roundings lie between an input and
an output or gradient (lookup, norm, send rows, two matmuls, activation, sum,
residual, and their gradients), added up: 12 x 2^-8 = 4.7e-2.
"""
import importlib.util
import os

import pytest
import torch

from tests._util import log

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
moe_layer = importlib.util.module_from_spec(spec)
spec.loader.exec_module(moe_layer)

TOL = 12 * 2.0 ** -8


def reference(p, ids, masks, douts, topk, coef, chosen):
    """The layer in float64; `chosen` are the experts that the GPU's router took
    (its logits come from rounded rows, so near ties may fall either way)."""
    leaf = {k: ([t.double().cpu().requires_grad_() for t in v] if isinstance(v, list) else
                v.double().cpu().requires_grad_()) for k, v in p.items()}
    table = torch.cat(leaf["tables"])
    w1, w2 = torch.cat(leaf["w1"]), torch.cat(leaf["w2"])
    experts = w1.shape[0]
    outs, total = [], 0.0
    for r in range(len(ids)):
        h = table[ids[r].cpu()]
        y = torch.nn.functional.layer_norm(h, h.shape[-1:], leaf["gamma"], leaf["beta"], 1e-5)
        prob = torch.softmax(y @ leaf["router"], 1)
        live = masks[r].cpu()
        n, at = int(live.sum()), chosen[r].cpu().long()
        gates = torch.gather(prob, 1, at.clamp(min=0)) * (at >= 0)
        gates = gates / gates.sum(1, keepdim=True).clamp(min=1e-30)
        rows = []
        for t in range(len(h)):
            out = torch.zeros_like(h[t])
            if live[t]:
                for j in range(topk):
                    z = y[t] @ w1[at[t, j]]
                    out = out + gates[t, j] * (torch.nn.functional.gelu(z, approximate="tanh") @ w2[at[t, j]])
            rows.append(out)
        out = torch.stack(rows) + h
        counts = torch.bincount(at[at >= 0], minlength=experts).double()
        total = total + (out * douts[r].double().cpu()).sum()
        total = total + coef * experts / (topk * n * n) * (counts * prob[live].sum(0)).sum()
        outs.append(out)
    total.backward()
    return outs, leaf


def near(got, want, what):
    got, want = got.double().cpu(), want.detach()
    err = float((got - want).norm() / want.norm())
    log(f"{what}: {err:.2e}")
    assert err <= TOL, f"{what}: normwise {err:.3e} > {TOL:.1e}"


def test_layer_step_matches_autograd():
    world, tokens, vocab, topk, pieces, coef = 2, 45, 96, 2, 2, 0.5
    p = moe_layer.make_params(world, vocab, 64, 96, 4)
    g = torch.Generator().manual_seed(3)
    ids = [torch.randint(0, vocab, (tokens,), generator=g).cuda() for _ in range(world)]
    masks = [(torch.rand(tokens, generator=g) > 0.2).cuda() for _ in range(world)]
    douts = [torch.randn(tokens, 64, generator=g).bfloat16().cuda() for _ in range(world)]
    outs, losses, state = moe_layer.forward(p, ids, masks, topk, pieces, coef)
    grads = moe_layer.backward(p, ids, masks, douts, coef, state)
    torch.cuda.synchronize()
    want, leaf = reference(p, ids, masks, douts, topk, coef, [r.ids for r in state[1]])
    for r in range(world):
        near(outs[r], want[r], f"rank {r}'s output")
        near(grads["tables"][r], leaf["tables"][r].grad, f"embedding shard {r}")
    for k in ("gamma", "beta", "router"):
        near(grads[k], leaf[k].grad, k)
