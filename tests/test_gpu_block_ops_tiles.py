"""The gated feed-forward block's products at sizes that take each tile and split, whole
and ragged, with enough of k to go round the tile's slots: whole numbers, whose sums
are exact, and random ones against float64."""
import numpy as np
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests._util import log
from tests.test_gpu_block_ops import act_bounds, guarded
from tests.test_gpu_block_ops_large import near_product
from tests.test_gpu_row_ops import HALF, TINY, equal, same_bits, within

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def numbers(seed, shape, least, most):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(least, most + 1, shape, generator=g, device="cuda").float()


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


# m, n, k; 16-bit results also have a tile of 256 x 256
@pytest.mark.parametrize("m,n,k", [
    (259, 27593, 656), (1300, 7001, 1040), (4095, 4090, 784), (1025, 13050, 400), (4000, 7001, 1040),   # 256 x 256
    (66, 18462, 1456), (2125, 65, 22544), (1406, 130, 14112), (65, 4241, 11280),        # 128 x 128, whole and split
    (2747, 135, 6944), (4196, 129, 6384),
    (33, 69, 704), (5905, 64, 4240), (33, 8339, 3232), (36, 73, 2416), (34, 67, 2192),  # 64 x 128, whole and split
    (35, 72, 1952), (33, 81, 2832), (39, 64, 3888),
])
def test_matmul_fp8_tiles(m, n, k):
    """Values to 2 and scales of 1/2 to 2: sums are multiples of 1/4 below 16 k < 2^19."""
    log(f"matmul_fp8 {m} x {n} x {k}")
    kb, nb = -(-k // 128), -(-n // 128)
    x, w = numbers(1, (m, k), -2, 2), numbers(2, (n, k), -2, 2)
    xs, ws = torch.exp2(numbers(3, (kb, m), -1, 1)), torch.exp2(numbers(4, (nb, kb), -1, 1))
    wide_x = x.double() * xs.t().repeat_interleave(128, 1)[:, :k]
    wide_w = w.double() * ws.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    ref = (wide_x @ wide_w.t().contiguous()).cpu().numpy()
    for dt, t in (("f32", torch.float32), ("bf16", torch.bfloat16), ("f16", torch.float16)):
        y, keep = guarded((m, n), t)
        tgc.matmul_fp8(x.to(F8), xs, w.to(F8), ws, y=y)
        torch.cuda.synchronize()
        keep("y")
        same_bits(y, ref, dt, dt)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("m,d,f", [
    (706, 392, 5544), (4093, 456, 1816), (1031, 1160, 3592),     # 256 x 256
    (200, 400, 4272), (339, 200, 2832),                          # 128 x 128, one a CU
    (525, 392, 3688), (199, 3208, 4152), (129, 4584, 2728), (66, 2984, 4104), (66, 3536, 2808),   # 128 x 128, two
    (33, 464, 72), (68, 2008, 2696), (65, 1688, 2064), (40, 1208, 64), (35, 976, 72), (41, 1976, 64),   # 64 x 128
])
def test_gated_ffn_tiles(m, d, f, kind):
    """The projections' sums are whole numbers up to 2 d."""
    log(f"gated ffn {m} x {d} x {f} {kind}")
    x, w = numbers(5, (m, d), -2, 2), numbers(6, (d, 2 * f), -1, 1)
    both = (x.double() @ w.double()).cpu().numpy()
    h, keep = guarded((m, f), torch.bfloat16)
    gate_up, keep_both = guarded((m, 2 * f), torch.bfloat16)
    tgc.gated_ffn(x.bfloat16(), w.bfloat16(), act=kind, h=h, gate_up=gate_up)
    torch.cuda.synchronize()
    keep("h")
    keep_both("gate_up")
    same_bits(gate_up, both, "bf16", "gate_up")
    off, ref = act_bounds(both, kind)
    within(h, ref, off * (1 + HALF["bf16"]) + HALF["bf16"] * np.abs(ref) + TINY["bf16"], "h")
    equal(h, tgc.gated_ffn(x.bfloat16(), w.bfloat16(), act=kind)[0], "h without saving")


@pytest.mark.parametrize("m,d,f", [
    (796, 5080, 400), (1094, 3600, 584), (2659, 2056, 1112),                # both products in 256 x 256
    (418, 3064, 72), (300, 1040, 1000), (435, 5160, 136), (606, 120, 72),   # 128 x 128 (one and two a CU), 64 x 128
    (2562, 96, 88), (33, 72, 1272), (33, 1288, 3104), (259, 3224, 2416),    # one by one, whole and split
    (1677, 72, 2648), (1931, 1352, 88),
])
def test_gated_ffn_backward_tiles(m, d, f):
    log(f"gated ffn backward {m} x {d} x {f}")
    x, w, dh, gate_up = normal(7, m, d), normal(8, d, 2 * f), normal(9, m, f), normal(10, m, 2 * f)
    dx, keep = guarded((m, d), torch.bfloat16)
    dw, keep_w = guarded((d, 2 * f), torch.bfloat16)
    tgc.gated_ffn_backward(dh, x, w, gate_up, act="gelu", dx=dx, dw=dw)
    torch.cuda.synchronize()
    keep("dx")
    keep_w("dw")
    dgu = tgc.gated_act_backward(dh, gate_up, act="gelu").double()
    near_product(dx, dgu, w.double().t().contiguous(), "dx")
    near_product(dw, x.double().t().contiguous(), dgu, "dw")
    equal(tgc.gated_ffn_backward(dh, x, w, gate_up, act="gelu", need_dw=False)[0], dx, "dx alone")
    equal(tgc.gated_ffn_backward(dh, x, w, gate_up, act="gelu", need_dx=False)[1], dw, "dw alone")
