"""Matrices close to 2^31 elements: what the gated block's kernels make of the last rows and
columns, and of sums over all rows, against the definitions."""
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests._util import log
from tests.test_gpu_block_ops import act_bounds
from tests.test_gpu_block_ops_large import filled, near_product
from tests.test_gpu_row_ops import HALF, TINY, U, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("m,d,f", [(1, 8184, 131064), (40, 8184, 131064), (200, 8184, 131064), (262136, 8184, 64)])
def test_gated_ffn_values_of_large_matrices(m, d, f, kind):
    """h of sampled rows and columns.  The projections are off by (2 (d + 8)) u of their terms;
    |act'| <= 1.13."""
    log(f"gated ffn {m} x {d} x {f} {kind}")
    x, w = filled((m, d), torch.bfloat16, 4), filled((d, 2 * f), torch.bfloat16, 5)
    w *= d ** -0.5
    h = tgc.gated_ffn(x, w, act=kind)[0]
    rows = torch.unique(torch.cat([torch.arange(min(m, 60)), torch.arange(max(0, m - 60), m)])).cuda()
    cols = torch.unique(torch.cat([torch.arange(min(f, 40)), torch.arange(f - 40, f)])).cuda()
    xr, wg, wu = x[rows].double(), w[:, cols].double().contiguous(), w[:, f + cols].double().contiguous()
    both, size = torch.cat([xr @ wg, xr @ wu], 1), torch.cat([xr.abs() @ wg.abs(), xr.abs() @ wu.abs()], 1)
    both, size, c = both.cpu().numpy(), size.cpu().numpy(), len(cols)
    off = (2 * (d + 8) + 4) * U * size
    bound, ref = act_bounds(both, kind)
    a = ref / both[:, c:]
    own = bound + 1.13 * off[:, :c] * (abs(both[:, c:]) + off[:, c:]) + abs(a) * off[:, c:]
    within(h[rows][:, cols], ref, own * (1 + HALF["bf16"]) + HALF["bf16"] * abs(ref) + TINY["bf16"], "h")


def test_gated_ffn_backward_of_a_large_x():
    """x, dx and their offsets close to 2^32 bytes; dw's sums run over all 262136 rows."""
    m, d, f = 262136, 8184, 64
    x, w = filled((m, d), torch.bfloat16, 4), filled((d, 2 * f), torch.bfloat16, 5)
    dh, gate_up = filled((m, f), torch.bfloat16, 6), filled((m, 2 * f), torch.bfloat16, 7)
    dx, dw = tgc.gated_ffn_backward(dh, x, w, gate_up)
    dgu = tgc.gated_act_backward(dh, gate_up)
    for rows in (slice(0, 60), slice(m - 60, m)):
        near_product(dx[rows], dgu[rows].double(), w.double().t().contiguous(), "dx")
    for cols in (slice(0, 40), slice(d - 40, d)):
        near_product(dw[cols], x[:, cols].double().t().contiguous(), dgu.double(), "dw")


def test_rms_norm_backward_of_many_rows():
    """dgamma's sums over 65535 rows of 32752, against float64 sums of chunks."""
    rows, n = 65535, 32752
    x = filled((rows, n), torch.float32)
    ga = torch.rand(n, device="cuda")
    rstd = torch.rand(rows, device="cuda") + 0.5
    dx, dgamma = tgc.rms_norm_backward(x, x, ga, rstd)
    ref, size = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    for r in range(0, rows, 2048):
        part = x[r:r + 2048].double().square() * rstd[r:r + 2048, None].double()
        ref += part.sum(0)
        size += part.abs().sum(0)
    # a product, up to 256 rows in one thread's sum, then 256 parts
    within(dgamma, ref.cpu().numpy(), (600 * U * size + U * ref.abs()).cpu().numpy(), "dgamma")
    for r in (slice(0, 30), slice(rows - 30, rows)):
        v, rs = x[r].double(), rstd[r, None].double()
        xh, g = v * rs, v * ga.double()
        want = rs * (g - xh * (g * xh).mean(1, keepdim=True))
        terms = rs * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
        within(dx[r], want.cpu().numpy(), (2 * 70 * U * terms + U * want.abs()).cpu().numpy(), "dx")
