"""Subnormal operands of the gated feed-forward block's products."""
import numpy as np
import pytest

import tensor_gemm_collective_amd as tgc
from tests.test_gpu_matmul_fp8_outliers import K, SIZES, TYPES, product_inputs
from tests.test_gpu_row_ops import HALF, gpu, same_bits, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", SIZES)
def test_matmul_fp8_of_subnormals(m, n):
    """e4m3's values below 2^-6, whole multiples of 2^-9: products to 49 steps of 2^-18, of which
    none lies below 2^-13 of another, and sums below 272 x 49 < 2^14 steps, all exact."""
    g = np.random.default_rng([m, n])
    x, w = g.integers(-7, 8, (m, K)) * 2.0 ** -9, g.integers(-7, 8, (n, K)) * 2.0 ** -9
    t = product_inputs(x, w)
    for dt in TYPES:
        # 2^12 brings the sums into fp16's normal range
        y = tgc.matmul_fp8(t[0], t[1] * 2.0 ** 12, t[2], t[3], dtype=TYPES[dt])
        same_bits(y, x @ w.T * 2.0 ** 12, dt, dt)


@pytest.mark.parametrize("m,f", [(1, 72), (40, 72), (300, 264), (1025, 2104), (4095, 4096)])
def test_gated_ffn_of_fp16_subnormals(m, f):
    """fp16 values below 2^-14 are whole multiples of 2^-24 and count as such: projections of
    up to 200 x 15 x 4 steps are exact."""
    g = np.random.default_rng([m, f])
    x, xv = gpu(g.integers(-15, 16, (m, 200)) * 2.0 ** -24, "f16")
    w, wv = gpu(g.integers(-4, 5, (200, 2 * f)), "f16")
    _, both = tgc.gated_ffn(x, w, save=True)
    same_bits(both, xv @ wv, "f16", "projections")


@pytest.mark.parametrize("m,f", [(1, 72), (40, 72), (300, 264), (1025, 2104), (4095, 4096)])
@pytest.mark.parametrize("ex,ew", [(-130, 100), (-100, -33), (-100, -40)])
def test_gated_ffn_of_bf16_subnormals(m, f, ex, ew):
    """Operands, sums and results below 2^-126: sums of up to 200 x 9 steps, exact in binary32
    (whose own steps end at 2^-149), and bf16's at 2^-133."""
    g = np.random.default_rng([m, f])
    x, xv = gpu(g.integers(-3, 4, (m, 200)) * 2.0 ** ex, "bf16")
    w, wv = gpu(g.integers(1, 4, (200, 2 * f)) * 2.0 ** ew, "bf16")
    _, both = tgc.gated_ffn(x, w, save=True)
    ref = xv @ wv
    within(both, ref, np.maximum(HALF["bf16"] * np.abs(ref), 2.0 ** -134), "projections")
