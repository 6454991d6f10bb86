"""Refusals of the row operators, on the host: the C entry points with
placeholder addresses (nothing may be enqueued, so these run only where no GPU
is visible), and the binding's checks of tensors."""
import ctypes

import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tensor_gemm_collective_amd import coc

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: host-only environment")

NULL, SPLIT, SHAPE, WORLD, DTYPE, ALIGN, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 6, 7, 9
G = 1 << 34   # placeholder addresses, 16 GiB apart


def at(i):
    return G * (i + 1)


LN = ["x", "residual", "gamma", "beta", "y", "sum_out", "mean", "rstd"]
LNB = ["dy", "x", "gamma", "mean", "rstd", "dsum", "dx", "dgamma", "dbeta"]
ROUTER = ["ids", "gates", "positions", "counts", "prob_sums", "loss", "valid"]


def ln(**kw):
    a = {k: at(i) for i, k in enumerate(LN)} | dict(rows=4, n=64, eps=1e-5, dt=2, pdt=2) | kw
    return tgc.lib().coc_layer_norm(*[a[k] for k in LN], a["rows"], a["n"], a["eps"], a["dt"], a["pdt"], None)


def lnb(**kw):
    a = {k: at(i) for i, k in enumerate(LNB)} | dict(rows=4, n=64, dt=2, pdt=0, ws=at(20), nws=1 << 20) | kw
    return tgc.lib().coc_layer_norm_backward(*[a[k] for k in LNB], a["rows"], a["n"], a["dt"], a["pdt"], a["ws"],
                                             a["nws"], None)


def emb(**kw):
    a = dict(ids=at(0), it=1, table=at(1), y=at(2), tokens=8, vocab=16, n=64, start=0, dt=2) | kw
    return tgc.lib().coc_embedding(a["ids"], a["it"], a["table"], a["y"], a["tokens"], a["vocab"], a["n"], a["start"],
                                   1.0, a["dt"], None)


def embg(**kw):
    a = dict(ids=at(0), it=1, dy=at(1), grad=at(2), tokens=8, vocab=16, n=64, start=0, acc=0, dt=2, gdt=0, ws=at(3),
             nws=1 << 20) | kw
    return tgc.lib().coc_embedding_grad(a["ids"], a["it"], a["dy"], a["grad"], a["tokens"], a["vocab"], a["n"],
                                        a["start"], 1.0, a["acc"], a["dt"], a["gdt"], a["ws"], a["nws"], None)


def router(**kw):
    a = {k: at(i + 2) for i, k in enumerate(ROUTER)} | dict(
        logits=at(0), ld=16, mask=at(1), tokens=8, experts=16, topk=2, pieces=4, world=8, dt=2, ws=at(20),
        nws=1 << 20) | kw
    return tgc.lib().coc_moe_router(a["logits"], a["ld"], a["mask"], *[a[k] for k in ROUTER], a["tokens"],
                                    a["experts"], a["topk"], a["pieces"], a["world"], 0.01, 1, a["dt"], a["ws"],
                                    a["nws"], None)


def routerb(**kw):
    names = ["mask", "ids", "gates", "counts", "valid", "dgates", "dloss", "dlogits"]
    a = {k: at(i + 1) for i, k in enumerate(names)} | dict(logits=at(0), ld=16, ldo=16, tokens=8, experts=16, topk=2,
                                                           pieces=4, dt=2) | kw
    return tgc.lib().coc_moe_router_backward(a["logits"], a["ld"], *[a[k] for k in names], a["ldo"], a["tokens"],
                                             a["experts"], a["topk"], a["pieces"], 0.01, 1, a["dt"], None)


def permute(**kw):
    a = dict(x=at(0), pos=at(1), out=at(2), tokens=8, rows=16, n=64, topk=2, dt=2) | kw
    return tgc.lib().coc_moe_permute(a["x"], a["pos"], a["out"], a["tokens"], a["rows"], a["n"], a["topk"], a["dt"],
                                     None)


def combine(**kw):
    a = dict(h=at(0), pos=at(1), gates=at(2), y=at(3), tokens=8, rows=16, n=64, topk=2, dt=2) | kw
    return tgc.lib().coc_moe_combine(a["h"], a["pos"], a["gates"], a["y"], a["tokens"], a["rows"], a["n"], a["topk"],
                                     a["dt"], None)


def combineb(**kw):
    names = ["dy", "h", "pos", "gates", "dh", "dgates"]
    a = {k: at(i) for i, k in enumerate(names)} | dict(tokens=8, rows=16, n=64, topk=2, dt=2) | kw
    return tgc.lib().coc_moe_combine_backward(*[a[k] for k in names], a["tokens"], a["rows"], a["n"], a["topk"],
                                              a["dt"], None)


CASES = [
    *[(ln, {k: None}, NULL) for k in LN if k not in ("residual", "beta")],
    (ln, dict(rows=-1), SHAPE), (ln, dict(n=0), SHAPE), (ln, dict(n=32769), SHAPE), (ln, dict(rows=1 << 26, n=1), SHAPE),
    (ln, dict(rows=1 << 25), SHAPE), (ln, dict(eps=-1.0), SHAPE), (ln, dict(eps=float("nan")), SHAPE),
    (ln, dict(dt=3), DTYPE), (ln, dict(dt=2, pdt=1), DTYPE), (ln, dict(dt=0, pdt=2), DTYPE),
    (ln, dict(x=at(0) + 1), ALIGN), (ln, dict(mean=at(6) + 2), ALIGN),
    (ln, dict(y=at(0)), ALIAS), (ln, dict(y=at(0) + 510), ALIAS), (ln, dict(sum_out=at(4) + 2), ALIAS),
    (ln, dict(rstd=at(6) + 12), ALIAS), (ln, dict(sum_out=at(1)), ALIAS),
    *[(lnb, {k: None}, NULL) for k in LNB if k not in ("dsum", "dbeta")],
    (lnb, dict(ws=None), WORKSPACE), (lnb, dict(nws=8), WORKSPACE), (lnb, dict(ws=at(20) + 2), ALIGN),
    (lnb, dict(dx=at(0)), ALIAS), (lnb, dict(ws=at(6)), ALIAS), (lnb, dict(dbeta=at(7) + 252), ALIAS),
    (lnb, dict(n=32769), SHAPE), (lnb, dict(pdt=1), DTYPE), (lnb, dict(rows=0, dgamma=None), NULL),
    *[(emb, {k: None}, NULL) for k in ("ids", "table", "y")],
    (emb, dict(it=2), DTYPE), (emb, dict(dt=-1), DTYPE), (emb, dict(n=0), SHAPE), (emb, dict(start=-1), SHAPE),
    (emb, dict(vocab=1 << 26, n=1), SHAPE), (emb, dict(tokens=1 << 25), SHAPE), (emb, dict(ids=at(0) + 4), ALIGN),
    (emb, dict(y=at(1) + 16), ALIAS), (emb, dict(y=at(0)), ALIAS),
    (emb, dict(n=1 << 30, tokens=1, vocab=1), SHAPE), (permute, dict(n=1 << 30, tokens=1, rows=1), SHAPE),
    *[(embg, {k: None}, NULL) for k in ("ids", "dy", "grad")],
    (embg, dict(ws=None), WORKSPACE), (embg, dict(nws=100), WORKSPACE), (embg, dict(ws=at(3) + 4), ALIGN),
    (embg, dict(gdt=1), DTYPE), (embg, dict(dt=0, gdt=2), DTYPE), (embg, dict(grad=at(1)), ALIAS),
    (embg, dict(ws=at(2)), ALIAS), (embg, dict(vocab=-1), SHAPE),
    *[(router, {k: None}, NULL) for k in ["logits"] + ROUTER],
    (router, dict(experts=0), SHAPE), (router, dict(experts=520, ld=520), SHAPE), (router, dict(topk=0), SHAPE),
    (router, dict(topk=17), SHAPE), (router, dict(experts=8, topk=9), SHAPE), (router, dict(ld=15), SHAPE),
    (router, dict(pieces=0), SPLIT), (router, dict(pieces=9), SPLIT), (router, dict(world=3), WORLD),
    (router, dict(world=16), WORLD), (router, dict(world=0), WORLD), (router, dict(dt=4), DTYPE),
    (router, dict(ws=None, tokens=100000), WORKSPACE), (router, dict(nws=16, tokens=100000), WORKSPACE), (router, dict(counts=at(5) + 4), ALIGN),
    (router, dict(gates=at(2) + 60), ALIAS), (router, dict(ids=at(0)), ALIAS),
    *[(routerb, {k: None}, NULL) for k in ("logits", "ids", "gates", "counts", "valid", "dlogits")],
    (routerb, dict(ldo=15), SHAPE), (routerb, dict(dlogits=at(0)), ALIAS), (routerb, dict(pieces=0), SPLIT),
    *[(permute, {k: None}, NULL) for k in ("x", "pos", "out")],
    (permute, dict(topk=17), SHAPE), (permute, dict(n=0), SHAPE), (permute, dict(out=at(0)), ALIAS),
    (permute, dict(x=at(0) + 1), ALIGN), (permute, dict(rows=-1), SHAPE),
    *[(combine, {k: None}, NULL) for k in ("h", "pos", "y")],
    (combine, dict(topk=0), SHAPE), (combine, dict(y=at(0) + 2), ALIAS), (combine, dict(dt=9), DTYPE),
    *[(combineb, {k: None}, NULL) for k in ("dy", "h", "pos", "gates", "dh", "dgates")],
    (combineb, dict(dh=at(1)), ALIAS), (combineb, dict(dgates=at(3)), ALIAS), (combineb, dict(tokens=-1), SHAPE),
]


@no_gpu_only
@pytest.mark.parametrize("fn,kw,status", CASES, ids=lambda v: getattr(v, "__name__", str(v)))
def test_entry_points_refuse(fn, kw, status):
    assert coc.STATUS[fn(**kw)] == coc.STATUS[status]
    assert tgc.lib().coc_last_error().decode() != ""


@no_gpu_only
def test_calls_without_rows_do_nothing():
    assert ln(rows=0, x=None, y=None) == 0
    assert emb(tokens=0, ids=None, y=None) == 0
    assert embg(vocab=0, grad=None) == 0
    assert embg(tokens=0, ids=None, dy=None, acc=1, ws=None) == 0
    assert routerb(tokens=0, logits=None) == 0
    assert permute(tokens=0) == 0 and permute(rows=0) == 0 and combine(tokens=0) == 0 and combineb(tokens=0) == 0


def test_workspace_sizes():
    L = tgc.lib()
    assert L.coc_layer_norm_backward_workspace_bytes(0, 64) == 0
    assert L.coc_layer_norm_backward_workspace_bytes(3, 64) >= 2 * 64 * 4
    assert L.coc_embedding_grad_workspace_bytes(0, 16, 64) == 0
    assert L.coc_embedding_grad_workspace_bytes(8, 16, 64) >= 8 * 8
    assert L.coc_moe_router_workspace_bytes(100, 16, 9) == 0
    assert L.coc_moe_router_workspace_bytes(100000, 16, 4) >= 4 * (16 * 8 + 4)


def _f(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call,error", [
    (lambda: tgc.layer_norm(_f(4, 8), _f(8)), ValueError),                                    # not on the GPU
    (lambda: tgc.layer_norm(_f(4, 8), _f(7)), ValueError),
    (lambda: tgc.layer_norm(_f(4, 8, dtype=torch.float64), _f(8)), TypeError),
    (lambda: tgc.layer_norm(_f(8), _f(8)), ValueError),
    (lambda: tgc.layer_norm(_f(8, 4).t(), _f(8)), ValueError),                                # not dense
    (lambda: tgc.layer_norm(_f(4, 8), _f(8), residual=_f(4, 8, dtype=torch.float16)), TypeError),
    (lambda: tgc.layer_norm(_f(4, 8), _f(8), _f(8, dtype=torch.float32)), TypeError),
    (lambda: tgc.layer_norm_backward(_f(4, 8), _f(4, 8), _f(8), _f(4), _f(4)), TypeError),    # statistics not fp32
    (lambda: tgc.embedding(_f(4), _f(8, 8)), TypeError),
    (lambda: tgc.embedding(_f(4, dtype=torch.int64), _f(8)), ValueError),
    (lambda: tgc.embedding_grad(_f(4, dtype=torch.int64), _f(3, 8), 8), ValueError),
    (lambda: tgc.embedding_grad(_f(4, dtype=torch.int64), _f(4, 8), 8, accumulate=True), ValueError),
    (lambda: tgc.moe_router(_f(8, 4).t(), 2), ValueError),
    (lambda: tgc.moe_router(_f(8, 4), 2, mask=_f(8)), TypeError),
    (lambda: tgc.moe_router(_f(8, 4), 2, mask=_f(7, dtype=torch.bool)), ValueError),
    (lambda: tgc.moe_permute(_f(8, 4), _f(8, 2, dtype=torch.int64)), TypeError),
    (lambda: tgc.moe_permute(_f(8, 4), _f(7, 2, dtype=torch.int32)), ValueError),
    (lambda: tgc.moe_combine(_f(16, 4), _f(8, 2, dtype=torch.int32), _f(8, 2)), TypeError),
    (lambda: tgc.moe_combine(_f(16, 4), _f(8, 2, dtype=torch.int32)), ValueError),            # not on the GPU
])
def test_binding_refuses(call, error):
    with pytest.raises(error):
        call()
