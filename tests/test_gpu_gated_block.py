"""examples/gated_block.py, a gated feed-forward block made of the library's
operators, against the same block in float64 with torch's autograd on the CPU.

Tolerance, normwise: every value that the block keeps in bf16 carries a rounding
of at most 2^-8 of itself; at most 10 such roundings lie between an input and an
output or gradient (sum, norm, projections, activation, partial and summed
product, and their gradients), added up: 10 x 2^-8 = 3.9e-2.  In 8 bits the two
products' operands carry one of at most 2^-4 each instead (a block's values are
at least 2^-6 of its largest, or count as little): 4 x 2^-4 at most, and by the
square root of their independent sum no more than sqrt(4) 2^-4 / sqrt(3) = 7.2e-2
with bf16's on top: 0.11.
"""
import importlib.util
import os

import pytest
import torch

from tests._util import log

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("gated_block", os.path.join(ROOT, "examples", "gated_block.py"))
gated_block = importlib.util.module_from_spec(spec)
spec.loader.exec_module(gated_block)

TOL, TOL8 = 10 * 2.0 ** -8, 0.11


def near(got, want, tol, what):
    err = float((got.double().cpu() - want).norm() / want.norm())
    assert err <= tol, f"{what}: {err:.2e}"


def reference(p, x, residual, act):
    """The block in float64 over all rows, with leaves for the gradients."""
    leaf = {k: ([t.double().cpu().requires_grad_() for t in v] if isinstance(v, list) else
                v.double().cpu().requires_grad_()) for k, v in p.items()}
    rows = torch.cat(x).double().cpu().requires_grad_()
    s = rows + torch.cat(residual).double().cpu()
    y = s * (s.square().mean(1, keepdim=True) + 1e-5).rsqrt() * leaf["gamma"]
    fn = torch.nn.functional.silu if act == "silu" else lambda t: torch.nn.functional.gelu(t, approximate="tanh")
    out, parts = 0.0, []
    for w, d in zip(leaf["w"], leaf["down"]):
        g, u = (y @ w).chunk(2, 1)
        parts.append((fn(g) * u) @ d)
        out = out + parts[-1]
    return leaf, rows, s, out, parts


def shards(world, tokens, hidden, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(tokens // world, hidden, generator=g).bfloat16().cuda() for _ in range(world)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("world", [1, 2, 4])
def test_gated_block_step(world, act):
    tokens, hidden, ffn = 256, 192, 512
    log(f"gated block over {world} ranks, {act}")
    p = gated_block.make_params(world, hidden, ffn)
    x, residual, douts, dsum = (shards(world, tokens, hidden, i) for i in range(4))
    outs, saved = gated_block.forward(p, x, residual, act)
    grads = gated_block.backward(p, douts, dsum, act, saved)
    leaf, rows, s, out, _ = reference(p, x, residual, act)
    ((out * torch.cat(douts).double().cpu()).sum() + (s * torch.cat(dsum).double().cpu()).sum()).backward()
    near(torch.cat(outs), out.detach(), TOL, "out")
    near(torch.cat(grads["rows"]), rows.grad, TOL, "d rows")
    near(grads["gamma"], leaf["gamma"].grad, TOL, "d gamma")
    for r in range(world):
        near(grads["w"][r], leaf["w"][r].grad, TOL, f"d w {r}")
        near(grads["down"][r], leaf["down"][r].grad, TOL, f"d down {r}")


@pytest.mark.parametrize("tokens", [1, 3, 20, 300])
def test_gated_block_in_8_bits(tokens):
    hidden, ffn = 400, 528
    p = gated_block.make_params(1, hidden, ffn)
    x, residual = shards(1, tokens, hidden, 5), shards(1, tokens, hidden, 6)
    got, total = gated_block.serve(p, gated_block.weights_fp8(p), x[0], residual[0], "silu")
    _, _, s, _, parts = reference(p, x, residual, "silu")
    near(got, parts[0].detach(), TOL8, "out")
    near(total, s.detach(), 2.0 ** -8, "residual")


def test_main_runs(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["gated_block.py", "--tokens", "128", "--hidden", "128", "--ffn", "256", "--steps", "2"])
    gated_block.main()
    assert "|out|" in capsys.readouterr().out
