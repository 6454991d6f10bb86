"""Plain fp64 definitions of the gated feed-forward block's operators: RMS norm,
gated activation and projections with their gradients, 8-bit values with scales
and their product.

Test infrastructure only (see oracle/__init__.py).  Each function is the
operator's formula (include/coc.h) in the plainest form; inputs are the storage
dtypes' values as float64, results are not rounded except to 8 bits.
"""
from __future__ import annotations

import numpy as np

BLOCK, TOP, LEAST = 128, 448.0, 2.0 ** -96


def rms_norm(h, gamma, eps):
    """(y, rstd) of the rows of h."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * gamma, rstd


def rms_norm_backward(dy, h, gamma, rstd, dsum=None):
    """(dx, dgamma) with the forward's statistic."""
    xh = h * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - xh * (g * xh).sum(1, keepdims=True) / h.shape[1])
    return (dx if dsum is None else dx + dsum), (dy * xh).sum(0)


# ------------------------------------------------------------------ 8 bits
def round_e4m3(x):
    """Nearest e4m3 values (ties to even) of x within [-448, 448]; three mantissa
    bits, exponents -6 to 8, steps of 2^-9 below 2^-6."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)                      # |x| in [2^(e-1), 2^e)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(x / step) * step         # rint: ties to even


def block_tops(y, block_rows):
    """The largest |y| of each block: (row blocks, column blocks)."""
    rows, n = y.shape
    out = np.zeros((-(-rows // block_rows), -(-n // BLOCK)))
    for r in range(out.shape[0]):
        for c in range(out.shape[1]):
            out[r, c] = np.abs(y[r * block_rows:(r + 1) * block_rows, c * BLOCK:(c + 1) * BLOCK]).max()
    return out


def quantize(y, block_rows):
    """(q, scales): the 8-bit values as float64, scales by (row block, column block)."""
    tops = np.maximum(block_tops(y, block_rows), LEAST)
    scales = tops / TOP
    return round_e4m3(y / spread(scales, block_rows, y.shape)), scales


def spread(scales, block_rows, shape):
    """Each value's scale."""
    return np.repeat(np.repeat(scales, block_rows, 0), BLOCK, 1)[:shape[0], :shape[1]]


def matmul_fp8(x, x_scales, w, w_scales):
    """x w^T of scaled values; x_scales by (column block, row), w_scales by (row
    block, column block), as the operators store them."""
    y = np.zeros((x.shape[0], w.shape[0]))
    for b in range(-(-x.shape[1] // BLOCK)):
        k = slice(b * BLOCK, (b + 1) * BLOCK)
        y += (x[:, k] * x_scales[b][:, None]) @ (w[:, k] * np.repeat(w_scales[:, b], BLOCK)[:w.shape[0], None]).T
    return y


# ------------------------------------------------------------------ gated block
def act(g, kind):
    """(act(g), act'(g))."""
    g = np.asarray(g, dtype=np.float64)
    c = np.sqrt(2.0 / np.pi)
    # gelu: (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)), which loses nothing far below zero
    z, dz = (g, 1.0) if kind == "silu" else (2 * c * (g + 0.044715 * g ** 3), 2 * c * (1.0 + 3 * 0.044715 * g * g))
    with np.errstate(over="ignore"):
        p, rest = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
    return g * p, p + g * p * rest * dz


def gated_act(gate_up, kind):
    f = gate_up.shape[1] // 2
    return act(gate_up[:, :f], kind)[0] * gate_up[:, f:]


def gated_act_backward(dh, gate_up, kind):
    f = gate_up.shape[1] // 2
    a, slope = act(gate_up[:, :f], kind)
    return np.concatenate([dh * gate_up[:, f:] * slope, dh * a], 1)


def gated_ffn(x, w, kind):
    """(h, gate_up)."""
    both = x @ w
    return gated_act(both, kind), both


def gated_ffn_backward(dh, x, w, gate_up, kind):
    """(dx, dw)."""
    d = gated_act_backward(dh, gate_up, kind)
    return d @ w.T, x.T @ d
