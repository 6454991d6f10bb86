"""The block's products over fewer stages of k than a tile has slots, as many, and one and
two more: each tile's start and end without the loop between them."""
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests._util import log
from tests.test_gpu_block_ops import guarded
from tests.test_gpu_block_ops_large import near_product
from tests.test_gpu_block_ops_tiles import numbers, normal
from tests.test_gpu_row_ops import same_bits

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.mark.parametrize("k", [16, 128, 144, 256, 272, 384, 528])
@pytest.mark.parametrize("m,n", [(1025, 13050), (4095, 4090),          # 16 bits: 256 x 256
                                 (2000, 4000),                         # 128 x 128
                                 (1300, 2600), (33, 69), (300, 2001),  # 64 x 128
                                 (24, 130)])
def test_matmul_fp8_of_short_rows(m, n, k):
    """Values to 2 and scales of 1/2 to 2: sums are multiples of 1/4, exact in binary32."""
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


@pytest.mark.parametrize("d", [8, 64, 72, 128, 136, 200, 264])
@pytest.mark.parametrize("m,f", [(4095, 4096), (1025, 13056),          # 256 x 256
                                 (2000, 2000), (700, 4096),            # 128 x 128
                                 (300, 4096), (500, 1000), (33, 72),   # 64 x 128, 128 x 128 with four slots
                                 (24, 1000)])
def test_gated_ffn_of_short_rows(m, f, d):
    log(f"gated ffn {m} x {d} x {f}")
    x, w = numbers(5, (m, d), -2, 2), numbers(6, (d, 2 * f), -1, 1)
    both = (x.double() @ w.double()).cpu().numpy()
    gate_up, keep = guarded((m, 2 * f), torch.bfloat16)
    tgc.gated_ffn(x.bfloat16(), w.bfloat16(), gate_up=gate_up)
    torch.cuda.synchronize()
    keep("gate_up")
    same_bits(gate_up, both, "bf16", "gate_up")


@pytest.mark.parametrize("m,d,f", [
    (1, 4096, 4096), (8, 4096, 4096), (65, 4096, 4096), (130, 4096, 4096), (200, 4096, 4096),   # dw: 256 x 256
    (1, 2048, 1024), (72, 2048, 1024), (136, 2048, 1024), (4, 600, 520), (90, 600, 520),        # smaller ones
    (4096, 4096, 8), (4096, 4096, 32), (4096, 4096, 72), (4096, 4096, 136), (2000, 520, 40),    # dx: few terms
])
def test_gated_ffn_backward_of_short_sums(m, d, f):
    log(f"gated ffn backward {m} x {d} x {f}")
    x, w, dh, gate_up = normal(7, m, d), normal(8, d, 2 * f), normal(9, m, f), normal(10, m, 2 * f)
    dx, keep = guarded((m, d), torch.bfloat16)
    dw, keep_w = guarded((d, 2 * f), torch.bfloat16)
    tgc.gated_ffn_backward(dh, x, w, gate_up, dx=dx, dw=dw)
    torch.cuda.synchronize()
    keep("dx")
    keep_w("dw")
    dgu = tgc.gated_act_backward(dh, gate_up).double()
    near_product(dx, dgu, w.double().t().contiguous(), "dx")
    near_product(dw, x.double().t().contiguous(), dgu, "dw")
