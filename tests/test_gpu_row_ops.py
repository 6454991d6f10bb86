"""GPU parity of the row operators against their fp64 definitions
(oracle/row_ops.py), at the sizes, masks and values where they can go wrong.

Tolerances.  u = 2^-24 bounds one binary32 rounding, `half(dt)` = eps / 2 the
rounding to the storage type (values that it holds exactly, or in one rounding
of a binary32 product, are compared bit for bit).  A sum of terms t_i along
paths of at most d additions is off by at most (d + 1) u sum|t_i|; each bound
below counts the longest path of any order a workgroup adds in (at most 32
values of a thread, 6 steps over a wave, 16 waves) and names the terms.
"""
import numpy as np
import pytest
import torch

import oracle
import tensor_gemm_collective_amd as tgc
from oracle import row_ops as R
from tests._util import TORCH_DT, encode_dtype, log, raw

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}   # least normal (f16: half its smallest step)
ROW = 32 + 6 + 16 + 10   # additions of a row's sum, and the operations around it


def gpu(a, dt):
    """float64 values rounded to `dt`, on the GPU; and the values they became."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TORCH_DT[dt]).cuda()
    return t, t.double().cpu().numpy()


def within(got, ref, bound, what):
    got = got.detach().double().cpu().numpy().reshape(np.shape(ref))
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} values off by more than the bound, the worst "
                           f"{np.max((err / np.maximum(bound, 1e-300))[bad]):.3g} times, first at {np.argwhere(bad)[0]}")


def same_bits(got, values, dt, what):
    a, b = raw(got).reshape(-1), encode_dtype(np.asarray(values, dtype=np.float64), dt).reshape(-1)
    if dt == "f32":
        a, b = a.view(np.uint32), b.astype(np.float32).view(np.uint32)
    assert np.array_equal(a, b), f"{what}: {(a != b).sum()} of {a.size} differ"


def equal(a, b, what):
    """Bit equality of two tensors (NaNs of equal bits included)."""
    assert a.dtype == b.dtype and a.shape == b.shape, what
    assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), what


# ------------------------------------------------------------------ layer norm
NORM = [  # rows, n, dtype, parameters' dtype, residual, beta
    (1, 1, "f32", "f32", False, True), (1, 7, "bf16", "bf16", False, True), (3, 64, "f16", "f32", True, True),
    (5, 513, "bf16", "f32", True, False), (2, 1027, "f16", "f16", False, True), (9, 2048, "bf16", "bf16", True, True),
    (7, 2049, "f32", "f32", True, True), (3, 4100, "bf16", "bf16", False, True), (2, 8192, "f16", "f16", True, True),
    (2, 8193, "bf16", "bf16", True, True), (1, 14336, "bf16", "bf16", False, True), (3, 16385, "f32", "f32", False, True),
    (2, 32768, "bf16", "bf16", True, True), (2, 32767, "f16", "f32", False, False), (301, 100, "bf16", "bf16", True, True),
    (1100, 33, "f32", "f32", False, True), (600, 4096, "bf16", "bf16", False, True),
]


def norm_inputs(rows, n, dt, pdt, residual, beta, seed=0, shift=0.25):
    g = np.random.default_rng([seed, rows, n])
    x = gpu(1.5 * g.standard_normal((rows, n)) + shift, dt)
    gamma, be = gpu(1 + 0.1 * g.standard_normal(n), pdt), gpu(0.1 * g.standard_normal(n), pdt)
    other = gpu(g.standard_normal((rows, n)), dt)
    return x, gamma, be if beta else (None, None), other if residual else (None, None), g


def check_norm(got, h, gamma, beta, eps, dt, what):
    y, mean, rstd = got
    ry, rm, rr = R.layer_norm(h, gamma, beta, eps)
    size = np.abs(h).mean(1)
    within(mean, rm, ROW * U * size, what + " mean")
    # the squares' sum, and the mean's error against the deviation in each square
    rel = 2 * ROW * U * (1 + size * rr)
    within(rstd, rr, rel * rr, what + " rstd")
    xh = np.abs(h - rm[:, None]) * rr[:, None]
    off = ((rel + 4 * U)[:, None] * xh + (ROW * U * size * rr)[:, None]) * np.abs(gamma) + 2 * U * np.abs(0 if beta is None else beta)
    within(y, ry, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ry) + TINY[dt], what + " y")


@pytest.mark.parametrize("case", NORM, ids=str)
def test_layer_norm(case):
    rows, n, dt, pdt, _, _ = case
    log(f"layer norm {case}")
    (x, xv), (ga, gav), (be, bev), (res, resv), _ = norm_inputs(*case)
    got = tgc.layer_norm(x, ga, be, residual=res, eps=1e-5)
    torch.cuda.synchronize()
    h = xv
    if res is not None:
        h = (xv.astype(np.float32) + resv.astype(np.float32)).astype(np.float64)
        same_bits(got[3], h, dt, "sum")
        h = got[3].double().cpu().numpy()
    check_norm(got[:3], h, gav, bev, 1e-5, dt, str(case))


@pytest.mark.parametrize("case", NORM, ids=str)
def test_layer_norm_backward(case):
    rows, n, dt, pdt, residual, _ = case
    log(f"layer norm backward {case}")
    (x, xv), (ga, gav), _, _, g = norm_inputs(*case)
    dy, dyv = gpu(g.standard_normal((rows, n)), dt)
    ds, dsv = gpu(g.standard_normal((rows, n)), dt) if residual else (None, None)
    mean = torch.from_numpy(xv.mean(1)).float().cuda()
    rstd = torch.from_numpy(1 / np.sqrt(xv.var(1) + 1e-5)).float().cuda()
    m, r = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    dx, dg, db = tgc.layer_norm_backward(dy, x, ga, mean, rstd, dsum=ds)
    again = tgc.layer_norm_backward(dy, x, ga, mean, rstd, dsum=ds)
    torch.cuda.synchronize()
    for a, b, what in zip((dx, dg, db), again, ("dx", "dgamma", "dbeta")):
        equal(a, b, f"{what} twice")
    rx, rg, rb = R.layer_norm_backward(dyv, xv, gav, m, r, dsv)
    xh, gg = (xv - m[:, None]) * r[:, None], dyv * gav
    terms = r[:, None] * (np.abs(gg) + np.abs(gg).mean(1, keepdims=True) +
                          np.abs(xh) * np.abs(gg * xh).mean(1, keepdims=True))
    off = 2 * ROW * U * terms + (U * np.abs(rx))
    within(dx, rx, off * (1 + HALF[dt]) + HALF[dt] * np.abs(rx) + TINY[dt], "dx")
    path = rows + 16
    for got, ref, t, what in ((dg, rg, np.abs(dyv * xh), "dgamma"), (db, rb, np.abs(dyv), "dbeta")):
        off = path * U * t.sum(0)
        within(got, ref, off * (1 + HALF[pdt]) + HALF[pdt] * np.abs(ref) + TINY[pdt], what)


def test_layer_norm_far_from_zero():
    """Mean 1000 times the deviation: the squares are taken of the distances."""
    (x, xv), (ga, gav), (be, bev), _, _ = norm_inputs(4, 5000, "f32", "f32", False, True, shift=1500.0)
    check_norm(tgc.layer_norm(x, ga, be, eps=1e-5), xv, gav, bev, 1e-5, "f32", "far")


def test_layer_norm_of_equal_and_bad_rows():
    """A row of one value is beta; NaN and infinities stay in their rows."""
    x = torch.randn(6, 777, device="cuda")
    x[1] = 3.0
    x[2, 5] = float("nan")
    x[3, 700] = float("inf")
    ga, be = torch.rand(777, device="cuda") + 0.5, torch.randn(777, device="cuda")
    y, mean, rstd = tgc.layer_norm(x, ga, be)
    assert torch.equal(y[1], be) and torch.isnan(y[2]).all() and not torch.isfinite(y[3]).any()
    good = [0, 4, 5]
    clean = tgc.layer_norm(x[good].contiguous(), ga, be)[0]
    equal(y[good], clean, "rows beside the bad ones")
    dx = tgc.layer_norm_backward(torch.ones_like(x), x, ga, mean, rstd)[0]
    assert torch.isfinite(dx[good]).all() and torch.isnan(dx[2]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_layer_norm_at_odd_addresses(dt):
    """Element-aligned views give the bits of 16-byte aligned tensors."""
    rows, n = 5, 1023
    (x, _), (ga, _), (be, _), (res, _), g = norm_inputs(rows, n, dt, dt, True, True)

    def odd(t):
        b = torch.empty(t.numel() + 3, dtype=t.dtype, device="cuda")[3:].view(t.shape)
        return b.copy_(t)

    want = tgc.layer_norm(x, ga, be, residual=res)
    got = tgc.layer_norm(odd(x), odd(ga), odd(be), residual=odd(res), y=odd(x))
    for a, b in zip(got, want):
        equal(a, b, "forward")
    dy = gpu(g.standard_normal((rows, n)), dt)[0]
    want = tgc.layer_norm_backward(dy, x, ga, want[1], want[2], dsum=res)
    got = tgc.layer_norm_backward(odd(dy), odd(x), odd(ga), odd(got[1]), odd(got[2]), dsum=odd(res))
    for a, b in zip(got, want):
        equal(a, b, "backward")


def test_layer_norm_backward_without_rows():
    z = torch.empty(0, 65, device="cuda")
    _, dg, db = tgc.layer_norm_backward(z, z, torch.ones(65, device="cuda"), z[:, 0].contiguous(), z[:, 0].contiguous(),
                                        dgamma=torch.ones(65, device="cuda"), dbeta=torch.ones(65, device="cuda"))
    assert not dg.any() and not db.any()


# ------------------------------------------------------------------ embedding
@pytest.mark.parametrize("tokens,vocab,n,dt", [(1, 1, 1, "f32"), (5, 7, 9, "bf16"), (300, 100, 515, "f16"),
                                               (33, 64, 4096, "bf16"), (2, 3, 20001, "f32"), (1000, 50, 8, "f16")])
def test_embedding(tokens, vocab, n, dt):
    log(f"embedding {tokens} {vocab} {n} {dt}")
    g = np.random.default_rng([7, tokens, n])
    table, tv = gpu(g.standard_normal((vocab, n)), dt)
    start, scale = 13, 1.7
    ids = g.integers(start - 3, start + vocab + 3, tokens)
    ids[0] = start + vocab - 1
    if tokens > 4:
        ids[1:5] = start - 1, start + vocab, -(2 ** 31), 2 ** 31 - 1
    want = R.embedding(ids, tv.astype(np.float32), start, np.float32(scale))
    want = np.where(want != 0, (tv.astype(np.float32) * np.float32(scale))[np.clip(ids - start, 0, vocab - 1)], 0.0)
    got = tgc.embedding(torch.from_numpy(ids).int().cuda(), table, start=start, scale=scale)
    same_bits(got, want, dt, "int32 ids")
    ids64 = torch.from_numpy(ids).long()
    if tokens > 4:
        ids64[3], ids64[4] = -(2 ** 63), 2 ** 63 - 1
    got = tgc.embedding(ids64.cuda(), table, start=start, scale=scale)
    same_bits(got, want, dt, "int64 ids")


GRADS = [  # tokens, vocab, n, dtype, gradient's dtype, ids
    (1, 1, 1, "f32", "f32", "any"), (1, 40, 65, "bf16", "bf16", "any"), (31, 5, 9, "f16", "f32", "any"),
    (32, 1, 64, "bf16", "f32", "one"), (33, 1, 64, "bf16", "bf16", "one"), (1000, 300, 515, "f32", "f32", "any"),
    (1024, 7, 40, "f16", "f16", "any"), (1025, 2000, 24, "bf16", "bf16", "skewed"), (5000, 60, 1100, "bf16", "bf16", "skewed"),
    (5000, 3, 129, "f32", "f32", "one"), (40000, 500, 16, "bf16", "f32", "skewed"), (40000, 90000, 3, "f16", "f16", "any"),
    (3000, 1100000, 2, "f32", "f32", "any"), (2048, 1500, 33, "bf16", "bf16", "skewed"),
    (10, 3000000, 1, "f32", "f32", "any"), (70, 50, 8, "bf16", "bf16", "none"), (2050, 10, 2056, "bf16", "bf16", "half"),
]


def grad_ids(kind, tokens, vocab, start, g):
    if kind == "one":
        return np.full(tokens, start + vocab // 2)
    if kind == "none":
        return np.full(tokens, start + vocab)
    if kind == "half":      # a batch padded with one id, to its half
        return np.where(np.arange(tokens) % 2, start, g.integers(start, start + vocab, tokens))
    if kind == "skewed":
        return start + np.floor(vocab ** g.random(tokens)).astype(np.int64) - 1
    return g.integers(start - 1, start + vocab + 1, tokens)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", GRADS, ids=str)
def test_embedding_grad(case, accumulate):
    tokens, vocab, n, dt, gdt, kind = case
    log(f"embedding grad {case} accumulate={accumulate}")
    g = np.random.default_rng([11, tokens, n])
    start, scale = 5, 0.75
    ids = grad_ids(kind, tokens, vocab, start, g)
    dy, dyv = gpu(g.standard_normal((tokens, n)), dt)
    old, oldv = gpu(g.standard_normal((vocab, n)), gdt)
    tid = torch.from_numpy(ids).cuda()
    grad = old.clone() if accumulate else torch.full_like(old, float("nan"))
    tgc.embedding_grad(tid, dy, vocab, start=start, scale=scale, grad=grad, accumulate=accumulate)
    again = old.clone() if accumulate else None
    again = tgc.embedding_grad(tid.int(), dy, vocab, start=start, scale=scale,
                               grad=again if accumulate else torch.empty_like(old), accumulate=accumulate)
    equal(grad, again, "twice")
    at = ids - start
    mine = (at >= 0) & (at < vocab)
    total, size, count = np.zeros((vocab, n)), np.zeros((vocab, n)), np.zeros(vocab)
    np.add.at(total, at[mine], dyv[mine])
    np.add.at(size, at[mine], np.abs(dyv[mine]))
    np.add.at(count, at[mine], 1)
    ref = scale * total + (oldv if accumulate else 0)
    off = (count[:, None] + 2) * U * scale * size + 2 * U * np.abs(ref)
    within(grad, ref, off * (1 + HALF[gdt]) + HALF[gdt] * np.abs(ref) + TINY[gdt], "gradient")
    rest = grad[torch.from_numpy(count == 0).cuda()]
    if accumulate:
        equal(rest, old[torch.from_numpy(count == 0).cuda()], "rows without tokens")
    else:
        assert not rest.any()


def test_embedding_grad_of_whole_numbers_is_exact():
    """Sums that binary32 holds exactly: every order gives these bits."""
    g = np.random.default_rng(3)
    ids = grad_ids("skewed", 9000, 300, 0, g)
    dyv = g.integers(-4, 5, (9000, 70)).astype(np.float64)
    got = tgc.embedding_grad(torch.from_numpy(ids).cuda(), gpu(dyv, "bf16")[0], 300, scale=0.5,
                             grad=torch.empty(300, 70, device="cuda"))
    same_bits(got, R.embedding_grad(ids, dyv, 300, 0, 0.5), "f32", "gradient")


def test_embedding_grad_keeps_nan_in_its_row():
    ids = torch.arange(200, device="cuda") % 20
    dy = torch.ones(200, 33, device="cuda")
    dy[45] = float("nan")
    got = tgc.embedding_grad(ids, dy, 21)
    assert torch.isnan(got[5]).all()
    good = [i for i in range(20) if i != 5]
    assert (got[good] == 10.0).all() and not got[20].any()


def test_embedding_without_tokens():
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert tgc.embedding(none, torch.ones(4, 8, device="cuda")).shape == (0, 8)
    assert not tgc.embedding_grad(none, torch.empty(0, 8, device="cuda"), 4,
                                  grad=torch.ones(4, 8, device="cuda")).any()


# ------------------------------------------------------------------ MoE router
ROUTERS = [  # tokens, experts, topk, pieces, world, dtype, mask
    (0, 8, 2, 2, 1, "f32", False), (1, 1, 1, 1, 1, "f32", False), (3, 2, 2, 8, 2, "bf16", False),
    (1, 16, 16, 1, 8, "f16", False), (5, 5, 3, 2, 5, "f32", True), (255, 9, 4, 1, 3, "bf16", False),
    (256, 8, 2, 4, 8, "f16", True), (257, 40, 5, 3, 8, "f32", True), (300, 16, 2, 4, 8, "f16", True),
    (1000, 64, 6, 2, 8, "bf16", True), (999, 100, 8, 7, 4, "f32", False), (2100, 128, 8, 2, 8, "bf16", False),
    (700, 200, 16, 5, 8, "f32", True), (513, 512, 8, 1, 8, "f16", True), (20000, 16, 2, 8, 8, "bf16", True),
    (18000, 4, 2, 1, 2, "f32", False),
]


def route_inputs(tokens, experts, topk, pieces, world, dt, masked, seed=0):
    g = np.random.default_rng([seed, tokens, experts])
    x, xv = gpu(1.3 * g.standard_normal((tokens, experts)) + 0.7 * g.standard_normal(experts), dt)
    mask = (g.random(tokens) >= 0.2).astype(np.uint8) if masked else None
    return x, xv, mask, None if mask is None else torch.from_numpy(mask).cuda(), g


def gate_bound(x, ids):
    """exp's argument is rounded once (u |x - max|); 32 roundings of the exp, sums and division."""
    far = np.abs(np.take_along_axis(x, np.maximum(ids, 0), 1) - x.max(1, keepdims=True))
    return (32 + np.minimum(far, 200)) * U


def check_routing(got, want, xv, what):
    for f in ("ids", "positions", "counts"):
        assert np.array_equal(getattr(got, f).cpu().numpy(), want[f]), f"{what}: {f}"
    assert int(got.valid) == want["valid"], what
    tokens = len(xv)
    if not tokens:
        assert float(got.loss) == 0.0 and not got.prob_sums.any()
        return
    with np.errstate(invalid="ignore"):
        b = np.where(want["ids"] >= 0, gate_bound(xv, want["ids"]), 0.0)
    within(got.gates, want["gates"], b * np.abs(want["gates"]) + TINY["f32"], f"{what}: gates")
    far = 32 + tokens + 40
    within(got.prob_sums, want["prob_sums"], far * U * want["prob_sums"] + tokens * TINY["f32"], f"{what}: sums")
    within(got.loss, np.array([want["loss"]]), (far + xv.shape[1]) * U * abs(want["loss"]) + TINY["f32"], f"{what}: loss")


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("case", ROUTERS, ids=str)
def test_router(case, renormalize):
    tokens, experts, topk, pieces, world, dt, masked = case
    log(f"router {case} renormalize={renormalize}")
    x, xv, mask, tmask, _ = route_inputs(*case)
    got = tgc.moe_router(x, topk, pieces=pieces, world=world, coef=0.02, renormalize=renormalize, mask=tmask)
    again = tgc.moe_router(x, topk, pieces=pieces, world=world, coef=0.02, renormalize=renormalize, mask=tmask)
    for a, b, f in zip(got, again, got._fields):
        equal(a, b, f"{f} twice")
    check_routing(got, R.moe_router(xv, topk, pieces, world, 0.02, renormalize, mask), xv, str(case))


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("case", [c for c in ROUTERS if c[0]], ids=str)
def test_router_backward(case, renormalize):
    tokens, experts, topk, pieces, world, dt, masked = case
    log(f"router backward {case} renormalize={renormalize}")
    x, xv, mask, tmask, g = route_inputs(*case)
    w = R.moe_router(xv, topk, pieces, world, 0.02, renormalize, mask)
    dg, dgv = gpu(g.standard_normal((tokens, topk)), "f32")
    dl, dlv = gpu(np.array([1.7 * tokens]), "f32")
    fwd = tgc.moe_router(x, topk, pieces=pieces, world=world, coef=0.02, renormalize=renormalize, mask=tmask)
    got = tgc.moe_router_backward(x, fwd.ids, fwd.gates, fwd.counts, fwd.valid, dg, dl, coef=0.02,
                                  renormalize=renormalize, mask=tmask)
    ref = R.moe_router_backward(xv, w["ids"], w["counts"], dgv, dlv[0], 0.02, renormalize, mask)
    p, live = R.softmax_rows(xv, mask)
    n = max(1, w["valid"])
    a = np.abs(dlv[0]) * 0.02 * experts / (topk * n * n) * w["counts"].sum(0)
    gd = np.abs(w["gates"] * dgv)
    own = np.zeros_like(p)
    np.put_along_axis(own, np.maximum(w["ids"], 0), gd * (w["ids"] >= 0), 1)
    if renormalize:     # g_j (d_j - sum g d): both terms; else the sum enters by p
        each = np.zeros_like(p)
        np.put_along_axis(each, np.maximum(w["ids"], 0), np.abs(w["gates"]) * (w["ids"] >= 0), 1)
        terms = p * (a + (p * a).sum(1, keepdims=True)) + own + each * gd.sum(1, keepdims=True)
    else:
        terms = p * (a + (p * a).sum(1, keepdims=True) + gd.sum(1, keepdims=True)) + own
    far = np.minimum(np.abs(xv - xv.max(1, keepdims=True)), 200)
    off = (80 + 2 * topk + 2 * far) * U * terms
    within(got, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], "dlogits")
    # each part alone
    part = tgc.moe_router_backward(x, fwd.ids, fwd.gates, fwd.counts, fwd.valid, None, dl, coef=0.02,
                                   renormalize=renormalize, mask=tmask)
    ref = R.moe_router_backward(xv, w["ids"], w["counts"], 0 * dgv, dlv[0], 0.02, renormalize, mask)
    within(part, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], "the loss alone")
    part = tgc.moe_router_backward(x, fwd.ids, fwd.gates, fwd.counts, fwd.valid, dg, None, coef=0.02,
                                   renormalize=renormalize, mask=tmask)
    ref = R.moe_router_backward(xv, w["ids"], w["counts"], dgv, 0.0, 0.02, renormalize, mask)
    within(part, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], "the gates alone")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_router_ties_empty_rows_and_bad_values(dt):
    """Ties go to the lowest index; rows of -inf and masked rows of anything take
    no part; rows with few logits above -inf choose only those."""
    inf, nan = float("inf"), float("nan")
    e = 12
    rows = [[0.0] * e, [1.0, 2.0] * 6, [-inf] * e, [-inf] * 11 + [-3.0], [-inf, 5.0] + [-inf] * 10,
            [nan] * e, [inf] * e, [-0.0, 0.0] * 6, [-100.0] * 3 + [60.0] + [-100.0] * 8, [nan, -inf] * 6,
            [torch.finfo(TORCH_DT[dt]).min] * e, [torch.finfo(TORCH_DT[dt]).max, 0.0] * 6]
    mask = np.ones(len(rows), dtype=np.uint8)
    mask[[5, 6, 9]] = 0
    x, xv = gpu(np.array(rows), dt)
    for renormalize in (False, True):
        got = tgc.moe_router(x, 4, pieces=3, world=2, coef=0.5, renormalize=renormalize,
                             mask=torch.from_numpy(mask).cuda().bool())
        want = R.moe_router(xv, 4, 3, 2, 0.5, renormalize, mask)
        for f in ("ids", "positions", "counts"):
            assert np.array_equal(getattr(got, f).cpu().numpy(), want[f]), f
        assert int(got.valid) == want["valid"] == 8
        within(got.gates, want["gates"], 64 * U * np.abs(want["gates"]) + TINY["f32"], "gates")
        within(got.loss, np.array([want["loss"]]), 200 * U * want["loss"], "loss")
        dx = tgc.moe_router_backward(x, got.ids, got.gates, got.counts, got.valid, torch.ones(len(rows), 4, device="cuda"),
                                     torch.ones(1, device="cuda"), coef=0.5, renormalize=renormalize,
                                     mask=torch.from_numpy(mask).cuda())
        assert torch.isfinite(dx).all() and not dx[[2, 5, 6, 9]].any()


def test_router_nan_of_a_live_token():
    x = torch.zeros(3, 6)
    x[1, 4] = float("nan")
    x[2, 3] = float("inf")
    got = tgc.moe_router(x.cuda(), 2)
    assert got.ids.tolist() == [[0, 1], [4, 0], [3, 0]]
    assert torch.isnan(got.loss).all() and torch.isnan(got.gates[1:]).all()
    assert torch.equal(got.gates[0].cpu(), torch.tensor([0.5, 0.5]))


def test_router_with_every_token_masked():
    got = tgc.moe_router(torch.randn(50, 8, device="cuda"), 2, pieces=2, world=2,
                         mask=torch.zeros(50, dtype=torch.bool, device="cuda"))
    assert (got.ids == -1).all() and (got.positions == -1).all() and not got.gates.any()
    assert not got.counts.any() and float(got.loss) == 0.0 and int(got.valid) == 0 and not got.prob_sums.any()


def test_router_of_strided_logits():
    """Logits padded to the matmul's width: the padding is neither read nor written."""
    wide = torch.randn(70, 24, device="cuda", dtype=torch.bfloat16)
    wide[:, 13:] = float("nan")
    x = wide[:, :13]
    a = tgc.moe_router(x, 3, pieces=2)
    b = tgc.moe_router(x.contiguous(), 3, pieces=2)
    for p, q, f in zip(a, b, a._fields):
        equal(p, q, f)
    dg, dl = torch.randn(70, 3, device="cuda"), torch.ones(1, device="cuda")
    out = torch.full((70, 24), 7.0, device="cuda", dtype=torch.bfloat16)
    tgc.moe_router_backward(x, a.ids, a.gates, a.counts, a.valid, dg, dl, dlogits=out[:, :13])
    want = tgc.moe_router_backward(x.contiguous(), a.ids, a.gates, a.counts, a.valid, dg, dl)
    equal(out[:, :13].contiguous(), want, "dlogits")
    assert (out[:, 13:] == 7.0).all()


# ------------------------------------------------------------------ MoE rows
ROWS = [  # tokens, n, topk, dtype, share of entries without a row
    (1, 1, 1, "f32", 0.0), (1, 14336, 2, "bf16", 0.0), (5, 7, 3, "f16", 0.4), (300, 130, 2, "f16", 0.0),
    (64, 2056, 8, "bf16", 0.2), (33, 4097, 4, "f32", 0.2), (9, 12288, 2, "bf16", 0.0), (1000, 64, 16, "bf16", 0.1),
    (2, 30001, 1, "f16", 0.0),
]


def row_inputs(tokens, n, topk, dt, without):
    g = np.random.default_rng([5, tokens, n])
    pos = g.permutation(tokens * topk).reshape(tokens, topk)
    pos[g.random(pos.shape) < without] = -1
    if tokens > 4:
        pos[3] = -1                     # a token without rows
        pos[4, 0] = tokens * topk + 5   # past the rows
    x, xv = gpu(g.standard_normal((tokens, n)), dt)
    h, hv = gpu(g.standard_normal((tokens * topk, n)), dt)
    ga, gav = gpu(g.random((tokens, topk)), "f32")
    return torch.from_numpy(pos).int().cuda(), pos, x, xv, h, hv, ga, gav


@pytest.mark.parametrize("case", ROWS, ids=str)
def test_permute(case):
    tokens, n, topk, dt, _ = case
    log(f"permute {case}")
    tp, pos, x, xv, *_ = row_inputs(*case)
    x.view(-1)[0] = float("nan")
    out = torch.full((tokens * topk, n), 9.0, dtype=x.dtype, device="cuda")
    tgc.moe_permute(x, tp, out=out)
    want = torch.full((tokens * topk, n), 9.0, dtype=x.dtype)
    for t in range(tokens):
        for r in pos[t]:
            if 0 <= r < tokens * topk:
                want[r] = x[t].cpu()
    equal(out.cpu(), want, "rows")


@pytest.mark.parametrize("case", ROWS, ids=str)
def test_combine(case):
    tokens, n, topk, dt, _ = case
    log(f"combine {case}")
    tp, pos, _, _, h, hv, ga, gav = row_inputs(*case)
    for gates, gv in ((ga, gav), (None, np.ones((tokens, topk)))):
        got = tgc.moe_combine(h, tp, gates)
        ref = R.moe_combine(hv, pos, gv)
        off = (topk + 1) * U * R.moe_combine(np.abs(hv), pos, gv)
        within(got, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], "sum")


@pytest.mark.parametrize("case", ROWS, ids=str)
def test_combine_backward(case):
    tokens, n, topk, dt, _ = case
    log(f"combine backward {case}")
    tp, pos, dy, dyv, h, hv, ga, gav = row_inputs(*case)
    dh = torch.full_like(h, 9.0)
    _, dg = tgc.moe_combine_backward(dy, h, tp, ga, dh=dh)
    rh, rg = R.moe_combine_backward(dyv, hv, pos, gav)
    named = np.zeros(tokens * topk, dtype=bool)
    named[pos[(pos >= 0) & (pos < tokens * topk)]] = True
    prod = np.full_like(rh, 9.0)
    for t in range(tokens):
        for j, r in enumerate(pos[t]):
            if 0 <= r < len(prod):
                prod[r] = gav[t, j].astype(np.float32) * dyv[t].astype(np.float32)
    same_bits(dh, prod, dt, "dh")
    size = R.moe_combine_backward(np.abs(dyv), np.abs(hv), pos, gav)[1]
    within(dg, rg, (n // 64 + 40) * U * size + TINY["f32"], "dgates")


def test_permute_and_its_gradient_are_adjoint():
    """<permute(x), r> = <x, combine(r)> in whole numbers, exactly."""
    tokens, n, topk = 50, 96, 3
    tp, pos, *_ = row_inputs(tokens, n, topk, "f32", 0.0)
    x = torch.randint(-4, 5, (tokens, n), device="cuda").float()
    r = torch.randint(-4, 5, (tokens * topk, n), device="cuda").float()
    out = tgc.moe_permute(x, tp, out=torch.zeros_like(r))
    assert (out * r).sum().item() == (x * tgc.moe_combine(r, tp)).sum().item()


# ------------------------------------------------------------------ offsets past 32 bits
def test_matrices_of_more_than_4_gib():
    """Rows whose bytes begin past 2^32, in every operator's big matrix."""
    rows, n = 131071, 16383                     # just below 2^31 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    line = torch.randn(2, n, generator=g, device="cuda")
    big = torch.zeros(rows, n, device="cuda")
    big[[70000, rows - 1]] = line
    ids = torch.tensor([rows - 1, 70000], device="cuda")
    equal(tgc.embedding(ids, big), line.flip(0).contiguous(), "lookup")
    pos = torch.tensor([[rows - 1], [70000]], dtype=torch.int32, device="cuda")
    equal(tgc.moe_combine(big, pos), line.flip(0).contiguous(), "combine")
    big.zero_()
    tgc.moe_permute(line, pos, out=big)
    equal(big[[rows - 1, 70000]], line, "permute")
    tgc.embedding_grad(ids, line, rows, grad=big)
    equal(big[[rows - 1, 70000]], line, "embedding gradient")
    assert not big[70001:rows - 1].any()
    del big
    x = torch.randn(65535, 32767, generator=g, device="cuda", dtype=torch.bfloat16)
    ga = torch.rand(32767, generator=g, device="cuda").bfloat16()
    y, mean, rstd = tgc.layer_norm(x, ga)
    want = tgc.layer_norm(x[-3:].contiguous(), ga)
    equal(y[-3:].contiguous(), want[0], "layer norm")
    dx = tgc.layer_norm_backward(x, x, ga, mean, rstd, dx=y)[0]
    want = tgc.layer_norm_backward(x[-3:].contiguous(), x[-3:].contiguous(), ga, mean[-3:].contiguous(),
                                   rstd[-3:].contiguous())[0]
    equal(dx[-3:].contiguous(), want, "layer norm backward")


# ------------------------------------------------------------------ streams and graphs
def whole_pass(s):
    """Every operator once, each on the one before's results."""
    emb = tgc.embedding(s["ids"], s["table"], scale=2.0)
    y, mean, rstd, h = tgc.layer_norm(emb, s["gamma"], s["beta"], residual=s["res"])
    r = tgc.moe_router(s["logits"], 2, pieces=2, world=2)
    rows = tgc.moe_permute(y, r.positions)
    out = tgc.moe_combine(rows, r.positions, r.gates)
    drows, dgates = tgc.moe_combine_backward(out, rows, r.positions, r.gates)
    dlogits = tgc.moe_router_backward(s["logits"], r.ids, r.gates, r.counts, r.valid, dgates, r.loss)
    dy = tgc.moe_combine(drows, r.positions)
    dx, dg, db = tgc.layer_norm_backward(dy, h, s["gamma"], mean, rstd, dsum=out)
    grad = tgc.embedding_grad(s["ids"], dx, len(s["table"]), scale=2.0)
    return [emb, y, mean, rstd, h, *r, rows, out, drows, dgates, dlogits, dy, dx, dg, db, grad]


def pass_state(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, n, v, e = 1500, 264, 90, 8
    f = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return {"ids": torch.randint(0, v, (t,), generator=g, device="cuda"), "table": f(v, n), "gamma": f(n), "beta": f(n),
            "res": f(t, n), "logits": f(t, e)}


def test_several_ops_in_one_graph():
    """A graph that holds every operator, replayed on changing inputs with eager
    calls between the replays: each replay gives the eager bits."""
    states = [pass_state(i) for i in range(3)]
    s = {k: v.clone() for k, v in states[0].items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        whole_pass(s)
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        outs = whole_pass(s)
    for i in (1, 0, 2, 1):
        for k in s:
            s[k].copy_(states[i][k])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = whole_pass(states[i])
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(outs, want)):
            equal(a, b, f"replay of state {i}, output {k}")


def test_calls_on_another_stream():
    """stream=: outputs and workspaces belong to it, whatever the current stream does meanwhile."""
    side = torch.cuda.Stream()
    dy = torch.randn(3000, 520, device="cuda")
    ids = torch.randint(0, 700, (3000,), device="cuda")
    ones = torch.ones(520, device="cuda")
    mean, rstd = dy.mean(1), dy.var(1).rsqrt()
    want = tgc.embedding_grad(ids, dy, 700)
    want_norm = tgc.layer_norm_backward(dy, dy, ones, mean, rstd)
    torch.cuda.synchronize()
    for _ in range(4):
        got = tgc.embedding_grad(ids, dy, 700, stream=side)
        norm = tgc.layer_norm_backward(dy, dy, ones, mean, rstd, stream=side)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]   # takes freed memory of this stream
        side.synchronize()
        equal(got, want, "embedding gradient")
        for a, b in zip(norm, want_norm):
            equal(a, b, "layer norm backward")
        del junk


# ------------------------------------------------------------------ with the all-to-all pair
def test_router_feeds_the_all_to_all():
    """counts and positions are what the MoE pair takes: dispatch and combine
    over one rank return every token's gate-weighted expert outputs."""
    t, hidden, ffn, e, k, pieces = 200, 64, 96, 4, 2, 2
    g = np.random.default_rng(9)
    x, xv = gpu(g.standard_normal((t, hidden)), "bf16")
    logits, _ = gpu(g.standard_normal((t, e)), "f32")
    w, wv = gpu(0.1 * g.standard_normal((e, hidden, ffn)), "bf16")
    r = tgc.moe_router(logits, k, pieces=pieces, world=1)
    rows = tgc.moe_permute(x, r.positions)
    counts = r.counts.cpu().numpy().reshape(pieces, 1, e)
    y, recv = tgc.alltoall_grouped_matmul(rows, [None], counts, w, 0)
    equal(recv, rows, "one rank's received rows are its send rows")
    out = tgc.moe_combine(y, r.positions, r.gates)
    ids, gates = r.ids.cpu().numpy(), r.gates.double().cpu().numpy()
    ref = np.zeros((t, ffn))
    size = np.zeros((t, ffn))
    for i in range(t):
        for j in range(k):
            ref[i] += gates[i, j] * (xv[i] @ wv[ids[i, j]])
            size[i] += gates[i, j] * (np.abs(xv[i]) @ np.abs(wv[ids[i, j]]))
    # the grouped matmul's rounding to bf16 under each gate, then the sum's
    within(out, ref, (hidden + 8) * U * size + 2 * HALF["bf16"] * np.abs(ref) + HALF["bf16"] * size, "layer")
