"""The 8-bit product where a few products are far above the others, or cancel."""
import numpy as np
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests._util import log
from tests.test_gpu_row_ops import HALF, same_bits, within

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# every kernel and tile of the 8-bit product; k of three blocks, the last one short
SIZES = [(1, 130), (9, 300), (24, 130), (100, 1000), (2000, 4000), (4095, 4090)]
K = 272


def product_inputs(x, w):
    """x, w (float64 values that e4m3 holds) and scales of 1."""
    kb = -(-x.shape[1] // 128)
    to8 = lambda v: torch.from_numpy(v).float().cuda().to(F8)  # noqa: E731
    return to8(x), torch.ones(kb, len(x), device="cuda"), to8(w), torch.ones(-(-len(w) // 128), kb, device="cuda")


@pytest.mark.parametrize("m,n", SIZES)
def test_matmul_fp8_of_outliers(m, n):
    """In every group of eight neighbouring k two products of 448 x 448, of one sign or of
    both, and six of 2 x 2.  All sums are multiples of 4 below 2^26, exact in binary32.
    Results in 16 bits may be off by 8 x 2^-13 of each group's largest product, here 196,
    and so need not hold the six at all; nothing else is lost but the last rounding."""
    log(f"matmul_fp8 of outliers {m} x {n}")
    g = np.random.default_rng([m, n])
    groups = K // 8
    x, w = np.full((m, K), 2.0), np.full((n, K), 2.0)
    first = 8 * np.arange(groups) + g.integers(0, 4, groups)
    second = first + g.integers(1, 5, groups)
    x[:, first] = x[:, second] = w[:, first] = 448.0
    w[:, second] = 448.0 * g.choice([-1.0, 1.0], (n, groups))
    t = product_inputs(x, w)
    ref = x @ w.T
    assert np.abs(x[0]) @ np.abs(w[0]) < 2 ** 26 and not (ref % 4).any()
    same_bits(tgc.matmul_fp8(*t, dtype=torch.float32), ref, "f32", "binary32")
    off = groups * 8 * 2.0 ** -13 * 448 * 448
    y = tgc.matmul_fp8(*t)
    within(y, ref, off * (1 + HALF["bf16"]) + HALF["bf16"] * np.abs(ref), "bf16")
    # fp16 holds results below 65504
    t = (*t[:3], t[3] / 4096)
    y = tgc.matmul_fp8(*t, dtype=torch.float16)
    within(y, ref / 4096, (off * (1 + HALF["f16"]) + HALF["f16"] * np.abs(ref)) / 4096, "f16")


@pytest.mark.parametrize("m,n", SIZES)
def test_matmul_fp8_of_one_outlier_that_cancels(m, n):
    """One group of 448 x 448, -448 x 448 and six products of 3.5 x 3.5: 73.5 in binary32; in 16
    bits within 8 x 2^-13 of the largest product of it."""
    x, w = np.zeros((m, K)), np.zeros((n, K))
    x[:, 40:48] = w[:, 40:48] = 3.5
    x[:, [41, 46]] = w[:, 41] = 448.0
    w[:, 46] = -448.0
    t = product_inputs(x, w)
    ref = np.full((m, n), 73.5)
    same_bits(tgc.matmul_fp8(*t, dtype=torch.float32), ref, "f32", "binary32")
    for dt in ("bf16", "f16"):
        off = 8 * 2.0 ** -13 * 448 * 448
        within(tgc.matmul_fp8(*t, dtype=TYPES[dt]), ref, off * (1 + HALF[dt]) + HALF[dt] * ref, dt)
