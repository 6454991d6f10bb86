"""examples/gated_block.py served in 8 bits over a group's ranks: the sum of their parts
against the block in float64.

Tolerance: each rank's part is off by at most the tolerance of one rank's block
(tests/test_gpu_gated_block.py), normwise and of its own size; the sum by these added
up, and a rounding to bf16 of each part and of the sum."""
import pytest
import torch

from tests._util import log
from tests.test_gpu_gated_block import TOL8, gated_block, near, reference, shards

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("world", [1, 2, 4])
@pytest.mark.parametrize("tokens", [1, 20, 300])
def test_gated_block_in_8_bits_over_a_group(tokens, world):
    hidden, ffn = 400, 64 * 4 * 5
    log(f"gated block in 8 bits, {tokens} tokens over {world} ranks")
    p = gated_block.make_params(world, hidden, ffn)
    x, residual = shards(1, tokens, hidden, 5), shards(1, tokens, hidden, 6)
    w8 = [gated_block.weights_fp8(p, r) for r in range(world)]
    got, total = gated_block.serve_group(p, w8, x[0], residual[0], "silu")
    _, _, s, out, parts = reference(p, x, residual, "silu")
    size = sum(float(t.detach().norm()) for t in parts)
    near(got, out.detach(), (TOL8 + 2 * 2.0 ** -8) * size / float(out.detach().norm()), "out")
    near(total, s.detach(), 2.0 ** -8, "residual")
    if world > 1:
        err = float((gated_block.serve(p, w8[0], x[0], residual[0], "silu")[0].double().cpu() - out.detach()).norm())
        assert err > 0.5 * float(out.detach().norm()), "one rank's part is not the sum"
