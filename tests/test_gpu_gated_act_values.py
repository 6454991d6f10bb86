"""The gated activation's binary32 rows where act(gate) is far below the gate."""
import numpy as np
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests.test_gpu_row_ops import U, gpu, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_act_of_far_gates_in_32_bits(kind):
    """act keeps its relative accuracy where it is tiny.  With e = exp(-|z|) (exp2 within one
    unit, 2 u, and its argument's remainder joined by a multiply-add) and r = 1 / (1 + e) (an
    addition, and a reciprocal within one unit): p, 1 - p within (3 + 3 + 1) u, act(g) u two
    products more, 9 u, taken as 12.  The slope adds p, as before, and g p (1 - p) z', with two
    more roundings of z' and three products: 24 u of it.  exp below 2^-126 counts as zero."""
    gate = np.concatenate([np.linspace(-80, 40, 24001) if kind == "silu" else np.linspace(-13, 13, 24001)])
    t, v = gpu(np.concatenate([gate, np.full_like(gate, 1.375)])[None], "f32")
    dh, dhv = gpu(np.full((1, len(gate)), 0.8125), "f32")
    gate, up = np.split(v, 2, 1)
    z, dz = (gate, 1.0) if kind == "silu" else (2 * np.sqrt(2 / np.pi) * (gate + 0.044715 * gate ** 3),
                                                2 * np.sqrt(2 / np.pi) * (1 + 0.134145 * gate ** 2))
    p, rest = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    least = 2.0 ** -126 * (1 + np.abs(gate)) * (1 + np.abs(z)) * 4
    a = gate * p
    within(tgc.gated_act(t, act=kind), a * up, 12 * U * np.abs(a * up) + least, "h")
    slope, part = p + a * rest * dz, 12 * U * p + 24 * U * np.abs(a * rest * dz) + U * np.abs(p + a * rest * dz)
    ref = np.concatenate([dhv * up * slope, dhv * a], 1)
    off = np.concatenate([dhv * up * (part + 3 * U * np.abs(slope)), 13 * U * np.abs(dhv * a)], 1)
    within(tgc.gated_act_backward(dh, t, act=kind), ref, off + np.tile(least, 2) * (1 + np.abs(z).max()), "dgate_up")
