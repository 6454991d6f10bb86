"""The router's results at logits far from zero, live and masked."""
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests._util import TORCH_DT, log
from tests.test_gpu_row_ops import equal

pytestmark = pytest.mark.gpu

FAR = [1e6, 3e7, 1e9, 3e9, 1e10, 1.1e10, 7e15, 1e20, 1e30, 9e36, 3e38]


def far_values(dt):
    """Values of either sign that `dt` holds, from where it rounds whole numbers to its largest."""
    top = torch.finfo(TORCH_DT[dt]).max
    return [s * v for v in [2e3, 6e4] + FAR if v <= top for s in (1.0, -1.0)]


@pytest.mark.parametrize("tokens,experts", [(48, 12), (3000, 12), (700, 128)])   # one workgroup; many
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_masked_logits_are_never_used(dt, tokens, experts):
    """Whatever a masked row holds, every output has the bits that zeros there give."""
    log(f"masked rows {dt} {tokens} x {experts}")
    g = torch.Generator().manual_seed(tokens)
    inf, nan = float("inf"), float("nan")
    x = torch.randn(tokens, experts, generator=g)
    mask = torch.arange(tokens) % 2 == 0
    clean = x.clone()
    clean[~mask] = 0.0
    at = 1
    while at < tokens:
        for v in far_values(dt) + [inf, -inf, nan]:
            for others in (v, 0.5 * v, 0.0):   # equal values; one far from the rest
                if at < tokens:
                    x[at] = others
                    x[at, at % experts] = v
                at += 2
    x, clean, mask = x.to(TORCH_DT[dt]).cuda(), clean.to(TORCH_DT[dt]).cuda(), mask.cuda()
    dg, dl = torch.randn(tokens, 3, generator=g).cuda(), torch.ones(1, device="cuda")
    for renormalize in (False, True):
        got = tgc.moe_router(x, 3, pieces=2, world=2, renormalize=renormalize, mask=mask)
        want = tgc.moe_router(clean, 3, pieces=2, world=2, renormalize=renormalize, mask=mask)
        assert torch.isfinite(want.prob_sums).all() and torch.isfinite(want.loss).all()
        for a, b, f in zip(got, want, got._fields):
            equal(a, b, f"{f}, renormalize={renormalize}")
        equal(tgc.moe_router_backward(x, got.ids, got.gates, got.counts, got.valid, dg, dl, renormalize=renormalize,
                                      mask=mask),
              tgc.moe_router_backward(clean, want.ids, want.gates, want.counts, want.valid, dg, dl,
                                      renormalize=renormalize, mask=mask), f"dlogits, renormalize={renormalize}")
