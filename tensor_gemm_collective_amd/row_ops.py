"""Binding of the row operators of include/coc.h: layer norm, embedding, MoE
router and MoE row moves, with their backward passes.

Argument marshalling only, as in coc.py.  Shapes, dtypes and devices are
checked here, where the tensors know them; sizes, alignment and overlap by the
library.  Outputs and workspaces are allocated where they are not given.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from .coc import _check, _dtype_code, _stream, lib

# torch's own quick way to the current stream's handle; current_stream() makes an
# object for it, which takes longer than a small kernel's launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_gpu(like):
    if not like.is_cuda:
        raise ValueError(f"the tensors must be on the GPU, got {like.device}")


def _new(shape, dtype, like, stream):
    """Memory for the work that goes to `stream`: allocated on that stream, so that
    the allocator neither hands out memory that earlier work of another stream still
    uses nor takes a workspace back before the call's kernels are done with it."""
    _on_gpu(like)
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _queue(stream, like):
    """The handle of the stream the call's work goes to."""
    _on_gpu(like)
    if like.device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {like.device}, the current device is {torch.cuda.current_device()}")
    if stream is None and _raw_stream is not None:
        return _raw_stream(like.device.index)
    return _stream(stream, like.device)


def _ptr(t):
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous (row-major)")
    return t.data_ptr()


def _want(t, name, like, dtype, *shape):
    """`t` is a dense tensor of that dtype and shape on like's device; returns its address."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return _ptr(t)


def _out(t, name, like, stream, dtype, *shape):
    if t is None:
        t = _new(shape, dtype, like, stream)
        return t, t.data_ptr()
    return t, _want(t, name, like, dtype, *shape)


def _opt(t, name, like, dtype, *shape):
    return None if t is None else _want(t, name, like, dtype, *shape)


def _workspace(ws, need, like, stream):
    """(tensor or None, address, bytes) of a workspace of at least `need` bytes."""
    if ws is None:
        if not need:
            return None, None, 0
        ws = _new(need, torch.uint8, like, stream)
    elif ws.device != like.device:
        raise ValueError(f"ws is on {ws.device}, expected {like.device}")
    return ws, _ptr(ws), ws.numel() * ws.element_size()


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    return t.shape


def layer_norm(x, gamma, beta=None, *, residual=None, eps=1e-5, y=None, sum_out=None, mean=None, rstd=None,
               stream=None):
    """Layer norm of the rows of x (rows x n), or of x + residual.

    gamma, beta: n values of x's dtype or float32.  Returns (y, mean, rstd), or
    (y, mean, rstd, sum) with a residual: sum is what was normalised, the next
    residual and the x of the backward pass."""
    rows, n = _matrix(x, "x")
    dt, pdt = _dtype_code(x), _dtype_code(gamma)
    px, pg = _ptr(x), _want(gamma, "gamma", x, gamma.dtype, n)
    pb = _opt(beta, "beta", x, gamma.dtype, n)
    pr = _opt(residual, "residual", x, x.dtype, rows, n)
    y, py = _out(y, "y", x, stream, x.dtype, rows, n)
    mean, pm = _out(mean, "mean", x, stream, torch.float32, rows)
    rstd, ps = _out(rstd, "rstd", x, stream, torch.float32, rows)
    po = None
    if residual is not None:
        sum_out, po = _out(sum_out, "sum_out", x, stream, x.dtype, rows, n)
    _check(lib().coc_layer_norm(px, pr, pg, pb, py, po, pm, ps, rows, n, eps, dt, pdt, _queue(stream, x)))
    return (y, mean, rstd) if residual is None else (y, mean, rstd, sum_out)


def layer_norm_backward(dy, x, gamma, mean, rstd, *, dsum=None, dx=None, dgamma=None, dbeta=None, ws=None,
                        stream=None):
    """Gradients of layer_norm by what it normalised (x: its input, or its sum),
    gamma and beta.  dsum (rows x n) is added to dx.  Returns (dx, dgamma, dbeta)."""
    rows, n = _matrix(x, "x")
    dt, pdt = _dtype_code(x), _dtype_code(gamma)
    pd, px = _want(dy, "dy", x, x.dtype, rows, n), _ptr(x)
    pg = _want(gamma, "gamma", x, gamma.dtype, n)
    pm, ps = _want(mean, "mean", x, torch.float32, rows), _want(rstd, "rstd", x, torch.float32, rows)
    pr = _opt(dsum, "dsum", x, x.dtype, rows, n)
    dx, po = _out(dx, "dx", x, stream, x.dtype, rows, n)
    dgamma, pdg = _out(dgamma, "dgamma", x, stream, gamma.dtype, n)
    dbeta, pdb = _out(dbeta, "dbeta", x, stream, gamma.dtype, n)
    L = lib()
    ws, pw, nw = _workspace(ws, L.coc_layer_norm_backward_workspace_bytes(rows, n), x, stream)
    _check(L.coc_layer_norm_backward(pd, px, pg, pm, ps, pr, po, pdg, pdb, rows, n, dt, pdt, pw, nw,
                                     _queue(stream, x)))
    return dx, dgamma, dbeta


def _ids_code(ids):
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    return 0 if ids.dtype == torch.int32 else 1


def embedding(ids, table, *, start=0, scale=1.0, y=None, stream=None):
    """scale * table[ids - start]; zeros for ids outside [start, start + len(table)).

    ids: any shape; returns ids.shape x n."""
    vocab, n = _matrix(table, "table")
    tokens, code = ids.numel(), _ids_code(ids)
    pi = _want(ids, "ids", table, ids.dtype, *ids.shape)
    y, py = _out(y, "y", table, stream, table.dtype, *ids.shape, n)
    _check(lib().coc_embedding(pi, code, _ptr(table), py, tokens, vocab, n, start, scale, _dtype_code(table),
                               _queue(stream, table)))
    return y


def embedding_grad(ids, dy, vocab, *, start=0, scale=1.0, grad=None, accumulate=False, ws=None, stream=None):
    """Gradient of embedding by its table of `vocab` rows, the sum over each row's
    tokens.  dy: ids.shape x n.  grad (vocab x n, dy's dtype or float32) is
    overwritten, or added to with accumulate."""
    n, tokens, code = dy.shape[-1], ids.numel(), _ids_code(ids)
    if accumulate and grad is None:
        raise ValueError("accumulate needs the gradient to add to")
    pi = _want(ids, "ids", dy, ids.dtype, *ids.shape)
    pd = _want(dy, "dy", dy, dy.dtype, *ids.shape, n)
    grad, pg = _out(grad, "grad", dy, stream, dy.dtype if grad is None else grad.dtype, vocab, n)
    L = lib()
    ws, pw, nw = _workspace(ws, L.coc_embedding_grad_workspace_bytes(tokens, vocab, n), dy, stream)
    _check(L.coc_embedding_grad(pi, code, pd, pg, tokens, vocab, n, start, scale, int(bool(accumulate)),
                                _dtype_code(dy), _dtype_code(grad), pw, nw, _queue(stream, dy)))
    return grad


class Routing(NamedTuple):
    """What moe_router returns; coc.h, coc_moe_router, defines each."""
    ids: object         # tokens x topk int32, -1: no choice
    gates: object       # tokens x topk float32
    positions: object   # tokens x topk int32, -1: no row
    counts: object      # pieces x experts int64
    prob_sums: object   # experts float32
    loss: object        # 1 float32
    valid: object       # 1 int64


def _logits(t, name):
    """(tokens, experts, row stride, address) of a matrix whose rows are dense."""
    tokens, experts = _matrix(t, name)
    if experts > 1 and tokens > 0 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be dense")
    ld = t.stride(0) if tokens > 1 else max(experts, 1)
    return tokens, experts, ld, t.data_ptr()


def _mask_ptr(mask, like, tokens):
    if mask is None:
        return None
    if mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    return _want(mask, "mask", like, torch.uint8, tokens)


def moe_router(logits, topk, *, pieces=1, world=1, coef=0.01, renormalize=True, mask=None, ids=None, gates=None,
               positions=None, counts=None, prob_sums=None, loss=None, valid=None, ws=None, stream=None):
    """Top-k routing of logits (tokens x experts, rows may be strided) with the
    per-expert counts, the rows' places in the send order and the balance loss.
    mask: tokens bool or uint8, 0 for tokens that take no part.  Returns a Routing."""
    tokens, experts, ld, pl = _logits(logits, "logits")
    pm = _mask_ptr(mask, logits, tokens)
    i32, f32, i64 = torch.int32, torch.float32, torch.int64
    ids, p0 = _out(ids, "ids", logits, stream, i32, tokens, topk)
    gates, p1 = _out(gates, "gates", logits, stream, f32, tokens, topk)
    positions, p2 = _out(positions, "positions", logits, stream, i32, tokens, topk)
    counts, p3 = _out(counts, "counts", logits, stream, i64, pieces, experts)
    prob_sums, p4 = _out(prob_sums, "prob_sums", logits, stream, f32, experts)
    loss, p5 = _out(loss, "loss", logits, stream, f32, 1)
    valid, p6 = _out(valid, "valid", logits, stream, i64, 1)
    L = lib()
    ws, pw, nw = _workspace(ws, L.coc_moe_router_workspace_bytes(tokens, experts, pieces), logits, stream)
    _check(L.coc_moe_router(pl, ld, pm, p0, p1, p2, p3, p4, p5, p6, tokens, experts, topk, pieces, world, coef,
                            int(bool(renormalize)), _dtype_code(logits), pw, nw, _queue(stream, logits)))
    return Routing(ids, gates, positions, counts, prob_sums, loss, valid)


def moe_router_backward(logits, ids, gates, counts, valid, dgates, dloss, *, coef=0.01, renormalize=True, mask=None,
                        dlogits=None, stream=None):
    """Gradient by the logits from the gates' (dgates) and the loss's (dloss, one
    float32 on the device); either may be None.  The other arguments are the
    forward's, and ids, gates, counts and valid its results."""
    tokens, experts, ld, pl = _logits(logits, "logits")
    topk, pieces = _matrix(ids, "ids")[1], _matrix(counts, "counts")[0]
    pm = _mask_ptr(mask, logits, tokens)
    i32, f32, i64 = torch.int32, torch.float32, torch.int64
    p0 = _want(ids, "ids", logits, i32, tokens, topk)
    p1 = _want(gates, "gates", logits, f32, tokens, topk)
    p2 = _want(counts, "counts", logits, i64, pieces, experts)
    p3 = _want(valid, "valid", logits, i64, 1)
    p4 = _opt(dgates, "dgates", logits, f32, tokens, topk)
    if dloss is not None:
        dloss = dloss.reshape(1)
    p5 = _opt(dloss, "dloss", logits, f32, 1)
    if dlogits is None:
        dlogits = _new((tokens, experts), logits.dtype, logits, stream)
    elif dlogits.dtype != logits.dtype or dlogits.shape != logits.shape or dlogits.device != logits.device:
        raise ValueError("dlogits must have the dtype, shape and device of logits")
    ld_out, po = _logits(dlogits, "dlogits")[2:]
    _check(lib().coc_moe_router_backward(pl, ld, pm, p0, p1, p2, p3, p4, p5, po, ld_out, tokens, experts, topk,
                                         pieces, coef, int(bool(renormalize)), _dtype_code(logits),
                                         _queue(stream, logits)))
    return dlogits


def moe_permute(x, positions, rows=None, *, out=None, stream=None):
    """out[positions[t, j]] = x[t].  rows: rows of out (default: one for each
    entry of positions); entries outside [0, rows) are skipped, and rows that
    no entry names are not written."""
    tokens, n = _matrix(x, "x")
    topk = _matrix(positions, "positions")[1]
    if rows is None:
        rows = tokens * topk if out is None else out.shape[0]
    pp = _want(positions, "positions", x, torch.int32, tokens, topk)
    out, po = _out(out, "out", x, stream, x.dtype, rows, n)
    _check(lib().coc_moe_permute(_ptr(x), pp, po, tokens, rows, n, topk, _dtype_code(x), _queue(stream, x)))
    return out


def moe_combine(h, positions, gates=None, *, y=None, stream=None):
    """y[t] = sum over j of gates[t, j] * h[positions[t, j]] (gates None: all 1,
    the gradient of moe_permute).  Entries outside h's rows are skipped."""
    rows, n = _matrix(h, "h")
    tokens, topk = _matrix(positions, "positions")
    pp = _want(positions, "positions", h, torch.int32, tokens, topk)
    pg = _opt(gates, "gates", h, torch.float32, tokens, topk)
    y, py = _out(y, "y", h, stream, h.dtype, tokens, n)
    _check(lib().coc_moe_combine(_ptr(h), pp, pg, py, tokens, rows, n, topk, _dtype_code(h),
                                 _queue(stream, h)))
    return y


def moe_combine_backward(dy, h, positions, gates, *, dh=None, dgates=None, stream=None):
    """Gradients of moe_combine: (dh, dgates).  Rows of dh that no entry of
    positions names are not written."""
    rows, n = _matrix(h, "h")
    tokens, topk = _matrix(positions, "positions")
    pd = _want(dy, "dy", h, h.dtype, tokens, n)
    pp = _want(positions, "positions", h, torch.int32, tokens, topk)
    pg = _want(gates, "gates", h, torch.float32, tokens, topk)
    dh, po = _out(dh, "dh", h, stream, h.dtype, rows, n)
    dgates, pdg = _out(dgates, "dgates", h, stream, torch.float32, tokens, topk)
    _check(lib().coc_moe_combine_backward(pd, _ptr(h), pp, pg, po, pdg, tokens, rows, n, topk, _dtype_code(h),
                                          _queue(stream, h)))
    return dh, dgates
