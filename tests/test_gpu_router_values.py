"""The router at values that a batch seldom holds: logits far from zero, live and
masked, and in its backward pass ids that are no expert's."""
import numpy as np
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from oracle import row_ops as R
from tests._util import TORCH_DT, log
from tests.test_gpu_row_ops import HALF, TINY, U, equal, gpu, within

pytestmark = pytest.mark.gpu

FAR = [1e6, 3e7, 1e9, 3e9, 1e10, 1.1e10, 7e15, 1e20, 1e30, 9e36, 3e38]


def far_values(dt):
    """Values of either sign that `dt` holds, from where it rounds whole numbers to its largest."""
    top = torch.finfo(TORCH_DT[dt]).max
    return [s * v for v in [2e3, 6e4] + FAR if v <= top for s in (1.0, -1.0)]


@pytest.mark.parametrize("tokens,experts", [(48, 12), (3000, 12), (700, 128)])   # one workgroup; many
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_masked_logits_are_never_used(dt, tokens, experts):
    """Whatever a masked row holds, every output has the bits that zeros there give."""
    log(f"masked rows {dt} {tokens} x {experts}")
    g = torch.Generator().manual_seed(tokens)
    inf, nan = float("inf"), float("nan")
    x = torch.randn(tokens, experts, generator=g)
    mask = torch.arange(tokens) % 2 == 0
    clean = x.clone()
    clean[~mask] = 0.0
    at = 1
    while at < tokens:
        for v in far_values(dt) + [inf, -inf, nan]:
            for others in (v, 0.5 * v, 0.0):   # equal values; one far from the rest
                if at < tokens:
                    x[at] = others
                    x[at, at % experts] = v
                at += 2
    x, clean, mask = x.to(TORCH_DT[dt]).cuda(), clean.to(TORCH_DT[dt]).cuda(), mask.cuda()
    dg, dl = torch.randn(tokens, 3, generator=g).cuda(), torch.ones(1, device="cuda")
    for renormalize in (False, True):
        got = tgc.moe_router(x, 3, pieces=2, world=2, renormalize=renormalize, mask=mask)
        want = tgc.moe_router(clean, 3, pieces=2, world=2, renormalize=renormalize, mask=mask)
        assert torch.isfinite(want.prob_sums).all() and torch.isfinite(want.loss).all()
        for a, b, f in zip(got, want, got._fields):
            equal(a, b, f"{f}, renormalize={renormalize}")
        equal(tgc.moe_router_backward(x, got.ids, got.gates, got.counts, got.valid, dg, dl, renormalize=renormalize,
                                      mask=mask),
              tgc.moe_router_backward(clean, want.ids, want.gates, want.counts, want.valid, dg, dl,
                                      renormalize=renormalize, mask=mask), f"dlogits, renormalize={renormalize}")


def far_rows(dt, experts, rows, g):
    """Rows around values far from zero: all equal, one above the rest by a step of the type, a few steps apart,
    and spread over the value's size to either side of zero."""
    out = []
    values = far_values(dt)
    t = TORCH_DT[dt]
    while len(out) < rows:
        v = float(torch.tensor(values[len(out) // 4 % len(values)]).to(t))
        step = torch.finfo(t).eps * abs(v)
        kind = len(out) % 4
        row = np.full(experts, v)
        if kind == 1:
            row -= step
            row[g.integers(experts)] += step
        elif kind == 2:
            row -= step * g.integers(0, 6, experts)
        elif kind == 3:
            row *= g.uniform(-1.0, 1.0, experts)
        out.append(row)
    x = torch.from_numpy(np.stack(out)).clamp(torch.finfo(t).min, torch.finfo(t).max).to(t)
    return x.cuda(), x.double().numpy()


def relative(xv, weights):
    """Relative errors of exp(x - top) / sum of weights * exp: the exponent's difference, its product with log2(e) and
    that constant are each off by a rounding, far = |x - top| of them; 40 roundings for the exponential, a sum over 64
    lanes of 8 and the quotient; and the divisor's own errors, which its terms weigh."""
    each = (40 + 4 * np.minimum(np.abs(xv - xv.max(1, keepdims=True)), 200)) * U
    return each + (weights * each).sum(1, keepdims=True)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("tokens,experts,topk", [(120, 12, 4), (1200, 12, 4), (600, 128, 8)])   # one workgroup; many
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_router_of_logits_far_from_zero(dt, tokens, experts, topk, renormalize):
    """Finite logits of any size, where log2(e) times the largest is rounded by more than an exponent's range."""
    log(f"far logits {dt} {tokens} x {experts} top {topk} renormalize={renormalize}")
    g = np.random.default_rng([tokens, experts])
    x, xv = far_rows(dt, experts, tokens, g)
    coef = 0.5
    got = tgc.moe_router(x, topk, pieces=2, world=2, coef=coef, renormalize=renormalize)
    want = R.moe_router(xv, topk, 2, 2, coef, renormalize)
    for f in ("ids", "positions", "counts"):
        assert np.array_equal(getattr(got, f).cpu().numpy(), want[f]), f
    assert int(got.valid) == want["valid"] == tokens
    ids, gates = want["ids"], want["gates"]
    p, _ = R.softmax_rows(xv)
    rel = relative(xv, p)
    under = np.zeros_like(p)
    np.put_along_axis(under, ids, gates, 1)
    grel = np.take_along_axis(relative(xv, under) if renormalize else rel, ids, 1)
    least = 2 * TINY["f32"]   # exponentials below it may be 0
    within(got.gates, gates, grel * gates + least, "gates")
    sums = (rel * p).sum(0) + tokens * (U * p.sum(0) + least)
    within(got.prob_sums, want["prob_sums"], sums, "prob_sums")
    counts = want["counts"].sum(0)
    scale = coef * experts / (topk * tokens * tokens)
    within(got.loss, np.array([want["loss"]]), scale * (counts * sums).sum() + (40 + experts) * U * want["loss"], "loss")

    dg, dgv = gpu(g.standard_normal((tokens, topk)), "f32")
    dl, dlv = gpu(np.array([1.7 * tokens]), "f32")
    dx = tgc.moe_router_backward(x, got.ids, got.gates, got.counts, got.valid, dg, dl, coef=coef,
                                 renormalize=renormalize)
    ref = R.moe_router_backward(xv, ids, want["counts"], dgv, dlv[0], coef, renormalize)
    # p_i (a_i - sum p a) + g_i (d_i - sum g d), or - p_i sum g d: each factor off by its relative error,
    # and the roundings of the products and sums
    a = np.abs(dlv[0]) * scale * counts
    pa = (p * a).sum(1, keepdims=True)
    gd = np.abs(gates * dgv)
    inner, inner_off = gd.sum(1, keepdims=True), (grel * gd).sum(1, keepdims=True)

    def spread(v):
        out = np.zeros_like(p)
        np.put_along_axis(out, ids, v, 1)
        return out

    terms = p * (a + pa) + spread(gd) + (spread(gates) if renormalize else p) * inner
    off = rel * p * (a + pa) + p * (rel * p * a).sum(1, keepdims=True) + spread(grel * gd)
    off += spread(gates * (grel * inner + inner_off)) if renormalize else p * (rel * inner + inner_off)
    off += (40 + 2 * topk) * U * terms + least * (2 + a.max() + 2 * np.abs(dgv).max() * topk)
    within(dx, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], "dlogits")


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts,topk", [(5, 3), (12, 4), (128, 8)])   # 1, 2 and 16 lanes a token
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_backward_takes_ids_of_no_expert_as_no_choice(dt, experts, topk, renormalize):
    tokens = 300
    log(f"ids of no expert {dt} {experts} top {topk} renormalize={renormalize}")
    g = torch.Generator().manual_seed(experts)
    x = torch.randn(tokens, experts, generator=g).to(TORCH_DT[dt]).cuda()
    r = tgc.moe_router(x, topk, renormalize=renormalize)
    bad = torch.tensor([experts, experts + 1, 8 * ((experts + 7) // 8), 513, 70000, 2 ** 31 - 1, -2, -2 ** 31],
                       dtype=torch.int32)
    ids, none = r.ids.cpu(), r.ids.cpu()
    for t in range(0, tokens, 3):
        ids[t, t % topk] = bad[t // 3 % len(bad)]
        none[t, t % topk] = -1
    ids[4], none[4] = bad[:topk].repeat(2)[:topk], -1
    dg, dl = torch.randn(tokens, topk, generator=g).cuda(), torch.ones(1, device="cuda")
    got = tgc.moe_router_backward(x, ids.cuda(), r.gates, r.counts, r.valid, dg, dl, renormalize=renormalize)
    want = tgc.moe_router_backward(x, none.cuda(), r.gates, r.counts, r.valid, dg, dl, renormalize=renormalize)
    equal(got, want, "dlogits")


@pytest.mark.parametrize("tokens,experts,topk,dt", [   # more tokens than a launch holds groups of lanes
    (70001, 64, 4, "f32"), (20003, 512, 8, "f32"), (20003, 300, 16, "bf16"), (70001, 128, 8, "f16"),
    (600001, 7, 2, "f32")])
def test_backward_of_many_tokens_is_that_of_its_pieces(tokens, experts, topk, dt):
    """A token's gradient depends on its own row and the batch's sums alone: tokens taken one after another by the
    same lanes have the bits that they have in calls of 997, where every token has its own."""
    log(f"router backward {tokens} x {experts} top {topk} {dt}")
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = (2 * torch.randn(tokens, experts, generator=g, device="cuda")).to(TORCH_DT[dt])
    mask = torch.rand(tokens, generator=g, device="cuda") > 0.1
    dg, dl = torch.randn(tokens, topk, generator=g, device="cuda"), torch.full((1,), 3.0 * tokens, device="cuda")
    for renormalize in (False, True):
        r = tgc.moe_router(x, topk, renormalize=renormalize, mask=mask)
        whole = tgc.moe_router_backward(x, r.ids, r.gates, r.counts, r.valid, dg, dl, renormalize=renormalize, mask=mask)
        for at in [a for a in range(0, tokens, 997) if a % 7 == 0 or a > tokens - 2000]:
            s = slice(at, at + 997)
            part = tgc.moe_router_backward(x[s], r.ids[s], r.gates[s], r.counts, r.valid, dg[s], dl,
                                           renormalize=renormalize, mask=mask[s])
            equal(whole[s].contiguous(), part, f"tokens {at} on, renormalize={renormalize}")
