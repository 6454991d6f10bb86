"""Binding of the gated feed-forward block's operators of include/coc.h: the
root-mean-square norm, the gated projections and activation with their backward
passes, and the matrix product in 8-bit floating point.

Argument marshalling only, as in coc.py.  Shapes, dtypes and devices are
checked here, where the tensors know them; sizes, alignment and overlap by the
library.  Outputs and workspaces are allocated where they are not given.

Values in 8 bits are torch.float8_e4m3fn tensors with float32 scales, one for
each 128 of a row: scales[b, row] (ceil(n / 128) x rows); or, for weights, one
for each 128 x 128: scales[r, b] (ceil(rows / 128) x ceil(n / 128)).
"""
from __future__ import annotations

import torch

from .coc import _check, _dtype_code, lib
from .row_ops import _matrix, _opt, _out, _ptr, _queue, _want, _workspace

_ACTS = {"silu": 0, "gelu": 1}
_FP8 = torch.float8_e4m3fn


def _act_code(act):
    if act not in _ACTS:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {act!r}")
    return _ACTS[act]


def _blocks(n):
    return (n + 127) // 128


def _halves(t, name):
    """(rows, f) of a rows x 2f matrix."""
    rows, both = _matrix(t, name)
    if both % 2:
        raise ValueError(f"{name} must have an even number of columns (gate, then up), got {both}")
    return rows, both // 2


def rms_norm(x, gamma, *, residual=None, eps=1e-5, y=None, sum_out=None, rstd=None, stream=None):
    """Root-mean-square norm of the rows of x (rows x n), or of x + residual.

    gamma: n values of x's dtype or float32.  Returns (y, rstd), or (y, rstd,
    sum) with a residual: sum is what was normalised, the next residual and the
    x of the backward pass."""
    rows, n = _matrix(x, "x")
    dt, pdt = _dtype_code(x), _dtype_code(gamma)
    px, pg = _ptr(x), _want(gamma, "gamma", x, gamma.dtype, n)
    pr = _opt(residual, "residual", x, x.dtype, rows, n)
    y, py = _out(y, "y", x, stream, x.dtype, rows, n)
    rstd, ps = _out(rstd, "rstd", x, stream, torch.float32, rows)
    po = None
    if residual is not None:
        sum_out, po = _out(sum_out, "sum_out", x, stream, x.dtype, rows, n)
    _check(lib().coc_rms_norm(px, pr, pg, py, po, ps, rows, n, eps, dt, pdt, _queue(stream, x)))
    return (y, rstd) if residual is None else (y, rstd, sum_out)


def rms_norm_fp8(x, gamma, *, residual=None, eps=1e-5, q=None, scales=None, sum_out=None, rstd=None, stream=None):
    """rms_norm with its output in 8 bits, a scale for each 128 of a row (n a
    multiple of 16).  Returns (q, scales, rstd), with a residual (q, scales,
    rstd, sum)."""
    rows, n = _matrix(x, "x")
    dt, pdt = _dtype_code(x), _dtype_code(gamma)
    px, pg = _ptr(x), _want(gamma, "gamma", x, gamma.dtype, n)
    pr = _opt(residual, "residual", x, x.dtype, rows, n)
    q, pq = _out(q, "q", x, stream, _FP8, rows, n)
    scales, pc = _out(scales, "scales", x, stream, torch.float32, _blocks(n), rows)
    rstd, ps = _out(rstd, "rstd", x, stream, torch.float32, rows)
    po = None
    if residual is not None:
        sum_out, po = _out(sum_out, "sum_out", x, stream, x.dtype, rows, n)
    _check(lib().coc_rms_norm_fp8(px, pr, pg, pq, pc, po, ps, rows, n, eps, dt, pdt, _queue(stream, x)))
    return (q, scales, rstd) if residual is None else (q, scales, rstd, sum_out)


def rms_norm_backward(dy, x, gamma, rstd, *, dsum=None, dx=None, dgamma=None, ws=None, stream=None):
    """Gradients of rms_norm by what it normalised (x: its input, or its sum) and
    gamma.  dsum (rows x n) is added to dx.  Returns (dx, dgamma)."""
    rows, n = _matrix(x, "x")
    dt, pdt = _dtype_code(x), _dtype_code(gamma)
    pd, px = _want(dy, "dy", x, x.dtype, rows, n), _ptr(x)
    pg, ps = _want(gamma, "gamma", x, gamma.dtype, n), _want(rstd, "rstd", x, torch.float32, rows)
    pr = _opt(dsum, "dsum", x, x.dtype, rows, n)
    dx, po = _out(dx, "dx", x, stream, x.dtype, rows, n)
    dgamma, pdg = _out(dgamma, "dgamma", x, stream, gamma.dtype, n)
    L = lib()
    ws, pw, nw = _workspace(ws, L.coc_rms_norm_backward_workspace_bytes(rows, n), x, stream)
    _check(L.coc_rms_norm_backward(pd, px, pg, ps, pr, po, pdg, rows, n, dt, pdt, pw, nw, _queue(stream, x)))
    return dx, dgamma


def quantize_fp8(x, *, block_rows=1, q=None, scales=None, stream=None):
    """x (rows x n, n a multiple of 16) in 8 bits, with a scale for each 128 of a
    row, or with block_rows=128 for each 128 x 128.  Returns (q, scales)."""
    rows, n = _matrix(x, "x")
    dt, px = _dtype_code(x), _ptr(x)
    shape = (_blocks(n), rows) if block_rows == 1 else (_blocks(rows), _blocks(n))
    q, pq = _out(q, "q", x, stream, _FP8, rows, n)
    scales, pc = _out(scales, "scales", x, stream, torch.float32, *shape)
    _check(lib().coc_quantize_fp8(px, pq, pc, rows, n, block_rows, dt, _queue(stream, x)))
    return q, scales


def matmul_fp8(x, x_scales, w, w_scales, *, dtype=torch.bfloat16, y=None, ws=None, stream=None):
    """x @ w.T of 8-bit operands: x m x k with a scale for each 128 of a row, w
    n x k with one for each 128 x 128.  y: m x n of `dtype`.  float32 has binary32
    sums; for 16-bit results the matrix units drop, in each group of eight
    neighbouring k, what lies below 2^-13 of the group's largest product."""
    m, k = _matrix(x, "x")
    n = _matrix(w, "w")[0]
    if x.dtype != _FP8:
        raise TypeError(f"x must be {_FP8}, got {x.dtype}")
    px, pxs = _ptr(x), _want(x_scales, "x_scales", x, torch.float32, _blocks(k), m)
    pw, pws = _want(w, "w", x, _FP8, n, k), _want(w_scales, "w_scales", x, torch.float32, _blocks(n), _blocks(k))
    y, py = _out(y, "y", x, stream, dtype if y is None else y.dtype, m, n)
    L = lib()
    ws, pk, nk = _workspace(ws, L.coc_matmul_fp8_workspace_bytes(m, n, k), x, stream)
    _check(L.coc_matmul_fp8(px, pxs, pw, pws, py, m, n, k, _dtype_code(y), pk, nk, _queue(stream, x)))
    return y


def gated_act(gate_up, *, act="silu", h=None, stream=None):
    """act(gate) * up of gate_up (rows x 2f, gate columns then up columns)."""
    rows, f = _halves(gate_up, "gate_up")
    code, dt, pg = _act_code(act), _dtype_code(gate_up), _ptr(gate_up)
    h, ph = _out(h, "h", gate_up, stream, gate_up.dtype, rows, f)
    _check(lib().coc_gated_act(pg, ph, rows, f, code, dt, _queue(stream, gate_up)))
    return h


def gated_act_fp8(gate_up, *, act="silu", q=None, scales=None, stream=None):
    """gated_act with its output in 8 bits, a scale for each 128 of a row (f a
    multiple of 16).  Returns (q, scales)."""
    rows, f = _halves(gate_up, "gate_up")
    code, dt, pg = _act_code(act), _dtype_code(gate_up), _ptr(gate_up)
    q, pq = _out(q, "q", gate_up, stream, _FP8, rows, f)
    scales, pc = _out(scales, "scales", gate_up, stream, torch.float32, _blocks(f), rows)
    _check(lib().coc_gated_act_fp8(pg, pq, pc, rows, f, code, dt, _queue(stream, gate_up)))
    return q, scales


def gated_act_backward(dh, gate_up, *, act="silu", dgate_up=None, stream=None):
    """Gradient of gated_act by gate_up."""
    rows, f = _halves(gate_up, "gate_up")
    code, dt, pg = _act_code(act), _dtype_code(gate_up), _ptr(gate_up)
    pd = _want(dh, "dh", gate_up, gate_up.dtype, rows, f)
    dgate_up, po = _out(dgate_up, "dgate_up", gate_up, stream, gate_up.dtype, rows, 2 * f)
    _check(lib().coc_gated_act_backward(pd, pg, po, rows, f, code, dt, _queue(stream, gate_up)))
    return dgate_up


def gated_ffn(x, w, *, act="silu", save=False, h=None, gate_up=None, ws=None, stream=None):
    """act(gate) * up with [gate up] = x @ w, formed together.  x: m x d; w: d x 2f,
    the gate columns and then the up columns.  Returns (h, gate_up); gate_up
    holds the projections where save asks for them or a tensor is given, and is
    None otherwise."""
    m, d = _matrix(x, "x")
    f = _halves(w, "w")[1]
    code, dt = _act_code(act), _dtype_code(x)
    px, pw = _ptr(x), _want(w, "w", x, x.dtype, d, 2 * f)
    h, ph = _out(h, "h", x, stream, x.dtype, m, f)
    pg = None
    if save or gate_up is not None:
        gate_up, pg = _out(gate_up, "gate_up", x, stream, x.dtype, m, 2 * f)
    L = lib()
    ws, pk, nk = _workspace(ws, L.coc_gated_ffn_workspace_bytes(m, d, f), x, stream)
    _check(L.coc_gated_ffn(px, pw, ph, pg, m, d, f, code, dt, pk, nk, _queue(stream, x)))
    return h, gate_up


def gated_ffn_backward(dh, x, w, gate_up=None, *, act="silu", need_dx=True, need_dw=True, dx=None, dw=None, ws=None,
                       stream=None):
    """Gradients of gated_ffn by x and w.  gate_up: what the forward saved, or
    None to compute the projections again.  Returns (dx, dw), None for one that
    is not needed."""
    m, d = _matrix(x, "x")
    f = _halves(w, "w")[1]
    code, dt = _act_code(act), _dtype_code(x)
    pd = _want(dh, "dh", x, x.dtype, m, f)
    px, pw = _ptr(x), _want(w, "w", x, x.dtype, d, 2 * f)
    pg = _opt(gate_up, "gate_up", x, x.dtype, m, 2 * f)
    po = pdw = None
    if need_dx:
        dx, po = _out(dx, "dx", x, stream, x.dtype, m, d)
    if need_dw:
        dw, pdw = _out(dw, "dw", x, stream, x.dtype, d, 2 * f)
    L = lib()
    ws, pk, nk = _workspace(ws, L.coc_gated_ffn_backward_workspace_bytes(m, d, f), x, stream)
    _check(L.coc_gated_ffn_backward(pd, px, pw, pg, po, pdw, m, d, f, code, dt, pk, nk, _queue(stream, x)))
    return dx if need_dx else None, dw if need_dw else None
