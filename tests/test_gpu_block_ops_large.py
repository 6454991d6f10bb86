"""The gated feed-forward block's operators on matrices close to 2^31 elements, at
offsets past 2^31 and 2^32 bytes: the rows' own results in a small call, bit for bit
where the same kernel runs, or against the definition."""
import numpy as np
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests._util import log
from tests.test_gpu_row_ops import equal

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def filled(shape, dtype, seed=1):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(seed))


def near_product(got, a, b, what):
    """got is a @ b (float64 on the GPU) summed in binary32 and rounded to bf16.  Values below
    2^-126, bf16's least normal number, may have been taken as zero, in an operand (which
    changes a term by at most 2^-126 times the other) or in the result."""
    k = a.shape[1]
    ref, size = a @ b, a.abs() @ b.abs()
    small = 2.0 ** -126 * (a.abs().sum(1)[:, None] + b.abs().sum(0)[None, :] + 1)
    off = 2 * (k + 8) * 2.0 ** -24 * size * 1.01 + 2.0 ** -8 * ref.abs() + small
    err = (got.double() - ref).abs()
    bad = ~(err <= off)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, {err[bad][0]} against {off[bad][0]} at {ref[bad][0]}"


def test_rms_norm_of_many_rows():
    rows, n = 65535, 32752
    x = filled((rows, n), torch.float32)
    ga = torch.rand(n, device="cuda")
    y, rstd = tgc.rms_norm(x, ga)
    last = x[-3:].contiguous()
    want = tgc.rms_norm(last, ga)
    for a, b, f in zip((y, rstd), want, ("y", "rstd")):
        equal(a[-3:].contiguous(), b, f)
    dx = tgc.rms_norm_backward(x, x, ga, rstd, dx=y)[0]
    equal(dx[-3:].contiguous(), tgc.rms_norm_backward(last, last, ga, want[1])[0], "dx")
    del y, dx
    q, s, _ = tgc.rms_norm_fp8(x, ga)
    q3, s3, _ = tgc.rms_norm_fp8(last, ga)
    equal(q[-3:].contiguous(), q3, "q")
    equal(s[:, -3:].contiguous(), s3, "scales")


def test_quantize_and_gated_act_of_many_rows():
    rows, n = 65535, 32736
    x = filled((rows, n), torch.float32)
    last = x[-3:].contiguous()
    for a, b in zip(tgc.quantize_fp8(x), tgc.quantize_fp8(last)):
        equal(a[-3:] if a.dtype == F8 else a[:, -3:].contiguous(), b, "quantize")
    q, s = tgc.quantize_fp8(x, block_rows=128)
    tail = x[-(rows % 128):].contiguous()
    q3, s3 = tgc.quantize_fp8(tail, block_rows=128)
    equal(q[-(rows % 128):], q3, "quantize blocks")
    equal(s[-1:].contiguous(), s3, "block scales")
    del q, s
    h = tgc.gated_act(x)
    equal(h[-3:].contiguous(), tgc.gated_act(last), "h")
    for a, b in zip(tgc.gated_act_fp8(x), tgc.gated_act_fp8(last)):
        equal(a[-3:] if a.dtype == F8 else a[:, -3:].contiguous(), b, "8 bits")
    d = tgc.gated_act_backward(h, x)
    equal(d[-3:].contiguous(), tgc.gated_act_backward(h[-3:].contiguous(), last), "dgate_up")


@pytest.mark.parametrize("m", [1, 9, 30, 100])
def test_matmul_fp8_of_a_large_weight(m):
    n, k = 262143, 8176
    log(f"matmul_fp8 {m} x {n} x {k}")
    w = torch.randint(0, 256, (n, k), dtype=torch.uint8, device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(2))
    w &= 0xB7   # no NaN, exponents spread
    w = w.view(F8)
    x, xs = tgc.quantize_fp8(filled((m, k), torch.float32))
    ws = torch.rand(2048, 64, device="cuda") + 0.5
    y = tgc.matmul_fp8(x, xs, w, ws, dtype=torch.float32)
    tail = n - 2047 * 128
    at = torch.cat([torch.arange(300), torch.arange(n - tail - 256, n)])
    wide = (x.float() * xs.repeat_interleave(128, 0)[:k].t()).double().cpu().numpy()
    for rows, blocks in ((slice(0, 256), slice(0, 2)), (slice(n - tail - 128, n), slice(2046, 2048))):
        part = w[rows].float().double().cpu().numpy()
        scale = np.repeat(np.repeat(ws[blocks].double().cpu().numpy(), 128, 0)[:len(part)], 128, 1)[:, :k]
        ref, size = wide @ (part * scale).T, np.abs(wide) @ np.abs(part * scale).T
        err = np.abs(y[:, rows].double().cpu().numpy() - ref)
        assert (err <= (2 * (k + 8) + 8) * 2.0 ** -24 * size).all(), f"{(err / size).max()}"
    assert torch.isfinite(y[:, at]).all()


def test_matmul_fp8_of_many_rows():
    m, k, n = 262143, 8176, 72
    x = torch.randint(0, 256, (m, k), dtype=torch.uint8, device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(3))
    x &= 0xB7
    x = x.view(F8)
    xs = torch.rand(64, m, device="cuda") + 0.5
    w, ws = tgc.quantize_fp8(filled((n, k), torch.float32), block_rows=128)
    y = tgc.matmul_fp8(x, xs, w, ws, dtype=torch.float32)
    wide = (w.float() * ws.repeat_interleave(128, 1)[:, :k]).double().cpu().numpy()
    part = (x[-100:].float() * xs[:, -100:].repeat_interleave(128, 0)[:k].t()).double().cpu().numpy()
    ref, size = part @ wide.T, np.abs(part) @ np.abs(wide).T
    err = np.abs(y[-100:].double().cpu().numpy() - ref)
    assert (err <= (2 * (k + 8) + 8) * 2.0 ** -24 * size).all(), f"{(err / size).max()}"


@pytest.mark.parametrize("m,d,f", [(1, 8184, 131064), (40, 8184, 131064), (200, 8184, 131064), (262136, 8184, 64)])
def test_gated_ffn_of_large_matrices(m, d, f):
    """w (then x) close to 2^31 elements of two bytes, forward and backward."""
    log(f"gated ffn {m} x {d} x {f}")
    x, w = filled((m, d), torch.bfloat16, 4), filled((d, 2 * f), torch.bfloat16, 5)
    h, both = tgc.gated_ffn(x, w, save=True)
    rows = slice(max(0, m - 50), m)
    cols = torch.cat([torch.arange(f - 40, f), torch.arange(2 * f - 40, 2 * f)]).cuda()
    near_product(both[rows][:, cols], x[rows].double(), w[:, cols].double().contiguous(), "projections")
    equal(tgc.gated_act(both[rows].contiguous())[:, -40:].isfinite(), h[rows][:, -40:].isfinite(), "h")
    if m > 200:
        return
    dx, dw = tgc.gated_ffn_backward(h, x, w, both)
    dgu = tgc.gated_act_backward(h, both)
    near_product(dx[rows, -40:], dgu[rows].double(), w[-40:].double().t().contiguous(), "dx")
    near_product(dw[-40:][:, cols], x[:, -40:].double().t().contiguous(), dgu[:, cols].double().contiguous(), "dw")
