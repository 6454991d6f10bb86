"""GPU parity of the gated feed-forward block's operators against their fp64
definitions (oracle/block_ops.py), at the sizes, masks and values where they can
go wrong.

Tolerances.  u = 2^-24 bounds one binary32 rounding, HALF[dt] = eps / 2 the
rounding to the storage type.  A sum of terms t_i along paths of at most d
additions is off by at most (d + 1) u sum|t_i| (twice that where the matrix unit
adds, which may cut off instead of rounding); each bound below counts the longest
path of any order.  exp2 and the reciprocal are good to 2^-22.
"""
import numpy as np
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from oracle import block_ops as B
from tests._util import log
from tests.test_gpu_row_ops import HALF, ROW, TINY, U, equal, gpu, same_bits, within

pytestmark = pytest.mark.gpu
HALF8 = 2.0 ** -4   # e4m3: half of 2^-3 relative, 2^-10 below 2^-6
F8 = torch.float8_e4m3fn


def guarded(shape, dtype):
    """(tensor, check): a tensor inside a larger one, and a check that what lies around it is as it was."""
    n = int(np.prod(shape))
    pad = 256
    big = torch.full((n + 2 * pad,), 7.0, device="cuda").to(dtype)
    before = big.clone()
    t = big[pad:pad + n].view(shape)

    def check(what):
        equal(big[:pad], before[:pad], what + ": memory in front of it")
        equal(big[pad + n:], before[pad + n:], what + ": memory behind it")
    return t, check


# ------------------------------------------------------------------ RMS norm
NORM = [  # rows, n, dtype, gamma's dtype, residual
    (1, 1, "f32", "f32", False), (1, 7, "bf16", "bf16", True), (3, 64, "f16", "f32", True), (5, 513, "bf16", "f32", True),
    (2, 1027, "f16", "f16", False), (9, 2048, "bf16", "bf16", True), (7, 2049, "f32", "f32", True),
    (3, 4100, "bf16", "bf16", False), (2, 8192, "f16", "f16", True), (2, 8193, "bf16", "bf16", True),
    (1, 14336, "bf16", "bf16", False), (3, 16385, "f32", "f32", False), (2, 32768, "bf16", "bf16", True),
    (2, 32767, "f16", "f32", False), (301, 100, "bf16", "bf16", True), (1100, 33, "f32", "f32", False),
    (600, 4096, "bf16", "bf16", False),
]
NORM8 = [c for c in NORM if c[1] % 16 == 0] + [(5, 16, "f32", "f32", True), (3, 144, "bf16", "f32", False),
                                               (17, 1040, "f16", "f16", True), (2, 4112, "f32", "f32", False)]


def norm_inputs(rows, n, dt, pdt, residual, seed=0):
    g = np.random.default_rng([seed, rows, n])
    x = gpu(1.5 * g.standard_normal((rows, n)), dt)
    gamma = gpu(1 + 0.1 * g.standard_normal(n), pdt)
    return x, gamma, gpu(g.standard_normal((rows, n)), dt) if residual else (None, None), g


def stored_sum(xv, resv, got, dt):
    if resv is None:
        return xv
    h = (xv.astype(np.float32) + resv.astype(np.float32)).astype(np.float64)
    same_bits(got, h, dt, "sum")
    return got.double().cpu().numpy()


def rms_bounds(h, gamma, y, rstd):
    """Of rstd (the squares' sum, a division, a root) and of y in binary32."""
    return ROW * U * rstd, (ROW + 4) * U * np.abs(y)


@pytest.mark.parametrize("case", NORM, ids=str)
def test_rms_norm(case):
    log(f"rms norm {case}")
    rows, n, dt, _, _ = case
    (x, xv), (ga, gav), (res, resv), _ = norm_inputs(*case)
    y, keep = guarded((rows, n), x.dtype)
    got = tgc.rms_norm(x, ga, residual=res, eps=1e-5, y=y)
    torch.cuda.synchronize()
    keep("y")
    h = stored_sum(xv, resv, got[2] if res is not None else None, dt)
    ry, rr = B.rms_norm(h, gav, 1e-5)
    off_r, off_y = rms_bounds(h, gav, ry, rr)
    within(got[1], rr, off_r, "rstd")
    within(y, ry, off_y * (1 + HALF[dt]) + HALF[dt] * np.abs(ry) + TINY[dt], "y")


def check_fp8(q, scales, y, off, block_rows, what):
    """Values and scales in 8 bits of y, which binary32 knows to `off`."""
    rows, n = y.shape
    s = scales.double().cpu().numpy()
    s = s.T if block_rows == 1 else s
    _, want = B.quantize(y, block_rows)
    # the largest value's own error, and two roundings
    within(torch.from_numpy(s), want, B.block_tops(off, block_rows) / 448 + 2 * U * want, what + " scales")
    wide = B.spread(s, block_rows, y.shape)
    got = q.double().cpu().numpy()
    assert np.abs(got).max(initial=0) <= 448
    # rounded from y (448 / top) with three roundings more; below 2^-6 in steps of 2^-9
    bound = (HALF8 * (1 + 8 * U) + 8 * U) * np.abs(y) + wide * 2.0 ** -10 + off * (1 + HALF8)
    within(torch.from_numpy(got * wide), y, bound, what + " values")


@pytest.mark.parametrize("case", NORM8, ids=str)
def test_rms_norm_fp8(case):
    log(f"rms norm fp8 {case}")
    rows, n, dt, _, _ = case
    (x, xv), (ga, gav), (res, resv), _ = norm_inputs(*case)
    q, keep = guarded((rows, n), F8)
    scales, keep_s = guarded((-(-n // 128), rows), torch.float32)
    got = tgc.rms_norm_fp8(x, ga, residual=res, q=q, scales=scales)
    again = tgc.rms_norm_fp8(x, ga, residual=res)
    torch.cuda.synchronize()
    keep("q")
    keep_s("scales")
    for a, b, what in zip(got, again, ("q", "scales", "rstd", "sum")):
        equal(a, b, what + " twice")
    h = stored_sum(xv, resv, got[3] if res is not None else None, dt)
    ry, rr = B.rms_norm(h, gav, 1e-5)
    off_r, off_y = rms_bounds(h, gav, ry, rr)
    within(got[2], rr, off_r, "rstd")
    check_fp8(q, scales, ry, off_y, 1, "rms norm")


@pytest.mark.parametrize("case", NORM, ids=str)
def test_rms_norm_backward(case):
    log(f"rms norm backward {case}")
    rows, n, dt, pdt, residual = case
    (x, xv), (ga, gav), _, g = norm_inputs(*case)
    dy, dyv = gpu(g.standard_normal((rows, n)), dt)
    ds, dsv = gpu(g.standard_normal((rows, n)), dt) if residual else (None, None)
    rstd = torch.from_numpy(1 / np.sqrt((xv ** 2).mean(1) + 1e-5)).float().cuda()
    r = rstd.double().cpu().numpy()
    dx, keep = guarded((rows, n), x.dtype)
    dx, dg = tgc.rms_norm_backward(dy, x, ga, rstd, dsum=ds, dx=dx)
    again = tgc.rms_norm_backward(dy, x, ga, rstd, dsum=ds)
    torch.cuda.synchronize()
    keep("dx")
    for a, b, what in zip((dx, dg), again, ("dx", "dgamma")):
        equal(a, b, f"{what} twice")
    rx, rg = B.rms_norm_backward(dyv, xv, gav, r, dsv)
    xh, gg = xv * r[:, None], dyv * gav
    terms = r[:, None] * (np.abs(gg) + np.abs(xh) * np.abs(gg * xh).mean(1, keepdims=True))
    off = 2 * ROW * U * terms + U * np.abs(rx)
    within(dx, rx, off * (1 + HALF[dt]) + HALF[dt] * np.abs(rx) + TINY[dt], "dx")
    off = (rows + 16) * U * np.abs(dyv * xh).sum(0)
    within(dg, rg, off * (1 + HALF[pdt]) + HALF[pdt] * np.abs(rg) + TINY[pdt], "dgamma")


def test_rms_norm_of_zero_and_bad_rows():
    """A row of zeros gives zeros; NaN and infinities stay in their rows (and in 8 bits in their blocks)."""
    x = torch.randn(6, 400, device="cuda")
    x[1] = 0.0
    x[2, 5] = float("nan")
    x[3, 390] = float("inf")
    ga = torch.rand(400, device="cuda") + 0.5
    y, rstd = tgc.rms_norm(x, ga)
    assert not y[1].any() and torch.isnan(y[2]).all() and torch.isnan(y[3, 390])
    good = [0, 1, 4, 5]
    equal(y[good], tgc.rms_norm(x[good].contiguous(), ga)[0], "rows beside the bad ones")
    q, s, _ = tgc.rms_norm_fp8(x, ga)
    equal(q[good], tgc.rms_norm_fp8(x[good].contiguous(), ga)[0], "rows beside the bad ones, 8 bits")
    assert not q[1].float().any() and torch.isfinite(s[:, good]).all() and torch.isnan(s[:, 2]).all()
    dx = tgc.rms_norm_backward(torch.ones_like(x), x, ga, rstd)[0]
    assert torch.isfinite(dx[good]).all() and torch.isnan(dx[2]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rms_norm_at_odd_addresses(dt):
    """Element-aligned views give the bits of 16-byte aligned tensors."""
    rows, n = 5, 1023
    (x, _), (ga, _), (res, _), g = norm_inputs(rows, n, dt, dt, True)

    def odd(t):
        b = torch.empty(t.numel() + 3, dtype=t.dtype, device="cuda")[3:].view(t.shape)
        return b.copy_(t)

    want = tgc.rms_norm(x, ga, residual=res)
    got = tgc.rms_norm(odd(x), odd(ga), residual=odd(res), y=odd(x))
    for a, b in zip(got, want):
        equal(a, b, "forward")
    dy = gpu(g.standard_normal((rows, n)), dt)[0]
    want = tgc.rms_norm_backward(dy, x, ga, want[1], dsum=res)
    got = tgc.rms_norm_backward(odd(dy), odd(x), odd(ga), odd(got[1]), dsum=odd(res))
    for a, b in zip(got, want):
        equal(a, b, "backward")
    x16, ga16 = x[:, :1008].contiguous(), ga[:1008].contiguous()
    for a, b in zip(tgc.rms_norm_fp8(odd(x16), odd(ga16)), tgc.rms_norm_fp8(x16, ga16)):
        equal(a, b, "8 bits")


def test_rms_norm_backward_without_rows():
    z = torch.empty(0, 65, device="cuda")
    _, dg = tgc.rms_norm_backward(z, z, torch.ones(65, device="cuda"), z[:, 0].contiguous(),
                                  dgamma=torch.ones(65, device="cuda"))
    assert not dg.any()


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("rows,n,dt,block_rows", [
    (1, 16, "f32", 1), (1, 16, "bf16", 128), (7, 144, "bf16", 1), (129, 272, "f16", 128), (300, 1040, "f32", 128),
    (33, 128, "f16", 1), (128, 128, "bf16", 128), (1000, 4112, "bf16", 1), (257, 2048, "f32", 1)])
def test_quantize(rows, n, dt, block_rows):
    g = np.random.default_rng([rows, n])
    x, xv = gpu(g.standard_normal((rows, n)) * np.exp2(g.integers(-8, 8, (rows, 1))), dt)
    q, keep = guarded((rows, n), F8)
    shape = (-(-n // 128), rows) if block_rows == 1 else (-(-rows // 128), -(-n // 128))
    scales, keep_s = guarded(shape, torch.float32)
    tgc.quantize_fp8(x, block_rows=block_rows, q=q, scales=scales)
    torch.cuda.synchronize()
    keep("q")
    keep_s("scales")
    check_fp8(q, scales, xv, np.zeros_like(xv), block_rows, "quantize")


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_edges(block_rows):
    """Blocks of zeros, of tiny and of the largest values, and with NaN and
    infinities, which come back as NaN without touching their neighbours."""
    x = torch.randn(256, 512, device="cuda")
    x[0:128, 0:128] = 0.0
    x[0:128, 128:256] = torch.randn(128, 128, device="cuda") * 2.0 ** -120
    x[0:128, 256:384] = 3.0e38
    x[200, 130] = float("nan")
    x[200, 300] = float("-inf")
    q, s = tgc.quantize_fp8(x, block_rows=block_rows)
    wide = s.t() if block_rows == 1 else s.repeat_interleave(128, 0)
    back = q.float() * wide.repeat_interleave(128, 1)
    assert not back[:128, :128].any() and not torch.signbit(q[:128, :128].float()).any()
    assert back[:128, 128:256].abs().max() < 2.0 ** -105
    assert ((back[:128, 256:384] / 3.0e38 - 1).abs() < 1e-6).all()
    bad = torch.zeros(256, 512, dtype=torch.bool, device="cuda")
    rows = slice(200, 201) if block_rows == 1 else slice(128, 256)
    bad[rows, 128:256] = True
    assert torch.isnan(back[rows, 128:256]).all()
    assert torch.isnan(back[rows, 256:384]).all() if block_rows == 1 else torch.isnan(back[200, 300])
    bad[rows, 256:384] = True
    assert torch.isfinite(back[~bad]).all()
    assert ((back - x)[~bad].abs() <= x[~bad].abs() * 0.07 + wide.repeat_interleave(128, 1)[~bad] * 2.0 ** -10).all()


# ------------------------------------------------------------------ the 8-bit product
PRODUCT = [  # m, n, k: every kernel and tile, ragged edges and short ends of k
    (1, 1, 16), (1, 129, 128), (2, 40, 1040), (4, 257, 2064), (5, 31, 272), (16, 300, 4112), (17, 130, 144), (32, 64, 2048),
    (33, 200, 1040), (64, 129, 400), (65, 1, 16), (100, 1000, 2064), (129, 257, 1168), (130, 140, 8192), (333, 1999, 1040),
    (300, 7168, 1040), (1, 7168, 8192), (9, 7168, 8208), (24, 2000, 8192), (1025, 3000, 528),
]


def fp8_operands(m, n, k, seed=0, ints=False):
    g = np.random.default_rng([seed, m, n, k])
    kb, nb = -(-k // 128), -(-n // 128)
    if ints:
        xv, wv = g.integers(-4, 5, (m, k)), g.integers(-4, 5, (n, k))
        xs, ws = np.exp2(g.integers(-2, 3, (kb, m))), np.exp2(g.integers(-2, 3, (nb, kb)))
    else:
        xv, wv = B.round_e4m3(g.standard_normal((m, k)) * 60), B.round_e4m3(g.standard_normal((n, k)) * 60)
        xs, ws = g.uniform(0.5, 2, (kb, m)) / 60, g.uniform(0.5, 2, (nb, kb)) / 60 / np.sqrt(k)
    to8 = lambda v: torch.from_numpy(v).float().cuda().to(F8)  # noqa: E731
    f32 = lambda v: torch.from_numpy(v).float().cuda()  # noqa: E731
    t = (to8(xv), f32(xs), to8(wv), f32(ws))
    return t, (xv.astype(float), t[1].double().cpu().numpy(), wv.astype(float), t[3].double().cpu().numpy())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", PRODUCT)
def test_matmul_fp8_of_whole_numbers(m, n, k, dt):
    """Small whole numbers with scales that are powers of two: every sum is exact."""
    log(f"matmul_fp8 {m} x {n} x {k} {dt}")
    t, v = fp8_operands(m, n, k, ints=True)
    y, keep = guarded((m, n), torch.float32 if dt == "f32" else torch.bfloat16)
    tgc.matmul_fp8(*t, y=y)
    torch.cuda.synchronize()
    keep("y")
    same_bits(y, B.matmul_fp8(*v), dt, "y")


@pytest.mark.parametrize("m,n,k", PRODUCT)
def test_matmul_fp8(m, n, k):
    """Binary32 results hold every product whole.  For 16-bit results the matrix unit adds
    groups of eight neighbouring k (the k of a lane in order) and drops bits below 2^-13 of
    the largest product's power of two: at most 8 x 2^-13 of that product a group."""
    log(f"matmul_fp8 {m} x {n} x {k}")
    t, (x, xs, w, ws) = fp8_operands(m, n, k, seed=1)
    ref = B.matmul_fp8(x, xs, w, ws)
    size = B.matmul_fp8(np.abs(x), xs, np.abs(w), ws)
    off = (2 * (k + 8) + 4) * U * size
    got = tgc.matmul_fp8(*t, dtype=torch.float32)
    again = tgc.matmul_fp8(*t, dtype=torch.float32)
    equal(got, again, "y twice")
    within(got, ref, off, "binary32")
    rows, cols = slice(None, None, max(1, m // 40)), slice(None, None, max(1, n // 60))
    wide = x[rows] * np.repeat(xs, 128, 0)[:k].T[rows], w[cols] * np.repeat(np.repeat(ws, 128, 0)[:n][cols], 128, 1)[:, :k]
    pad = -(-k // 8) * 8 - k
    ga, gb = (np.abs(np.pad(a, ((0, 0), (0, pad)))).reshape(len(a), -1, 8) for a in wide)
    group = sum((ga[:, None, :, :][:, :, c:c + 16] * gb[None, :, :, :][:, :, c:c + 16]).max(-1).sum(-1)
                for c in range(0, ga.shape[1], 16))
    for dt in ("bf16", "f16"):
        y = tgc.matmul_fp8(*t, dtype=torch.bfloat16 if dt == "bf16" else torch.float16)
        e = off[rows][:, cols] + 2.0 ** -10 * group
        r = ref[rows][:, cols]
        within(y[rows][:, cols], r, e * (1 + HALF[dt]) + HALF[dt] * np.abs(r) + TINY[dt], dt)


def test_matmul_fp8_keeps_bad_values_in_their_rows():
    """NaN in a row of x, or in a scale, reaches that row alone; and no row reads another's."""
    for m in (3, 40, 200):
        t, _ = fp8_operands(m, 300, 400, seed=2)
        want = tgc.matmul_fp8(*t)
        x, xs = t[0].clone(), t[1].clone()
        x.view(torch.uint8)[1, 399] = 0x7F
        xs[3, 2] = float("nan")
        got = tgc.matmul_fp8(x, xs, *t[2:])
        assert torch.isnan(got[1:3]).all()
        keep = [i for i in range(m) if i not in (1, 2)]
        equal(got[keep], want[keep], "other rows")


def test_matmul_fp8_without_k():
    z = torch.empty(3, 0, device="cuda").to(F8)
    y = torch.ones(3, 5, device="cuda")
    tgc.matmul_fp8(z, torch.empty(0, 3, device="cuda"), z[:1].expand(5, 0).contiguous(), torch.empty(1, 0, device="cuda"),
                   y=y)
    assert not y.any()


# ------------------------------------------------------------------ gated activation
def gate_values(g, rows, f):
    v = 2 * g.standard_normal((rows, 2 * f))
    v.reshape(-1)[::max(1, v.size // 40)] *= 12   # some far out
    return v


def act_bounds(gate_up, kind):
    """(bound of h, h): the exponent's argument rounds a few times, the rest to 2^-22 each."""
    f = gate_up.shape[1] // 2
    g, u = gate_up[:, :f], gate_up[:, f:]
    z = np.abs(g) if kind == "silu" else 1.6 * np.abs(g + 0.044715 * g ** 3)
    h = B.gated_act(gate_up, kind)
    p = 1 / (1 + np.exp(np.minimum(np.where(g < 0, z, -z), 700)))   # about act(g) / g
    rel = (8 * np.minimum(z, 800) * (1 - p) + 16) * U * 4
    return rel * np.abs(h) + 2.0 ** -126 * (np.abs(u) + 1) * (np.abs(g) + 1), h


ACT = [(1, 1, "f32"), (3, 5, "bf16"), (2, 8, "f16"), (7, 129, "f32"), (301, 100, "bf16"), (5, 4099, "f16"), (40, 3584, "bf16"),
       (1000, 3, "f16")]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("rows,f,dt", ACT)
def test_gated_act(rows, f, dt, kind):
    log(f"gated act {rows} x {f} {dt} {kind}")
    g = np.random.default_rng([rows, f])
    t, v = gpu(gate_values(g, rows, f), dt)
    dh, dhv = gpu(g.standard_normal((rows, f)), dt)
    h, keep = guarded((rows, f), t.dtype)
    d, keep_d = guarded((rows, 2 * f), t.dtype)
    tgc.gated_act(t, act=kind, h=h)
    tgc.gated_act_backward(dh, t, act=kind, dgate_up=d)
    torch.cuda.synchronize()
    keep("h")
    keep_d("dgate_up")
    off, ref = act_bounds(v, kind)
    within(h, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], "h")
    ref = B.gated_act_backward(dhv, v, kind)
    # p (1 - p) changes by its own size per unit of the argument, whose rounding is as above;
    # the slope's two parts each carry it
    gate = v[:, :f]
    z = np.abs(gate) if kind == "silu" else 1.6 * np.abs(gate + 0.044715 * gate ** 3)
    p = 1 / (1 + np.exp(np.minimum(np.where(gate < 0, z, -z), 700)))
    inner = 1 if kind == "silu" else 1.6 * (1 + 0.134145 * np.minimum(np.abs(gate), 20) ** 2)
    part = p + np.abs(gate) * p * (1 - p) * inner
    rel = (8 * np.minimum(z, 800) + 32) * U * 4
    slope = rel * part + 2.0 ** -24 * 4 * np.abs(gate) * p * inner
    off = np.concatenate([np.abs(dhv * v[:, f:]) * slope, np.abs(dhv) * np.abs(gate) * p * rel], 1) + 2.0 ** -120 * (
        1 + np.abs(np.concatenate([dhv * v[:, f:], dhv], 1)))
    within(d, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], "dgate_up")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("rows,f,dt", [(1, 16, "f32"), (5, 144, "bf16"), (33, 1040, "f16"), (300, 3584, "bf16"), (17, 272, "f32")])
def test_gated_act_fp8(rows, f, dt, kind):
    g = np.random.default_rng([rows, f])
    t, v = gpu(gate_values(g, rows, f), dt)
    q, keep = guarded((rows, f), F8)
    scales, keep_s = guarded((-(-f // 128), rows), torch.float32)
    tgc.gated_act_fp8(t, act=kind, q=q, scales=scales)
    torch.cuda.synchronize()
    keep("q")
    keep_s("scales")
    off, ref = act_bounds(v, kind)
    check_fp8(q, scales, ref, off, 1, "gated act")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_act_of_far_values(kind):
    """Gates of any size: act is the gate or zero, its slope one or zero; NaN stays NaN."""
    gate = torch.tensor([[-3e38, -1e20, -200.0, -0.0, 0.0, 200.0, 1e20, 3e38, float("nan")]], device="cuda")
    one = torch.ones_like(gate)
    t = torch.cat([gate, one], 1)
    h = tgc.gated_act(t, act=kind)
    want = torch.where(gate > 1, gate, 0.0)
    assert torch.equal(h[0, :8], want[0, :8]) and torch.isnan(h[0, 8])
    d = tgc.gated_act_backward(one, t, act=kind)
    slope = torch.where(gate > 1, 1.0, torch.where(gate.abs() < 1, 0.5, 0.0))
    assert torch.equal(d[0, :8], slope[0, :8]) and torch.equal(d[0, 9:17], want[0, :8])
    assert torch.isnan(d[0, 8]) and torch.isnan(d[0, 17])


# ------------------------------------------------------------------ gated projections
FFN = [  # m, d, f, dtype: every tile, split and unsplit, ragged edges and short ends of k
    (1, 8, 8, "bf16"), (1, 8192, 3584, "bf16"), (3, 72, 40, "f16"), (16, 1000, 136, "bf16"), (17, 64, 8, "f16"),
    (32, 520, 264, "bf16"), (33, 200, 72, "bf16"), (64, 2056, 64, "f16"), (100, 512, 128, "bf16"), (129, 72, 1000, "f16"),
    (200, 8192, 256, "bf16"), (300, 1040, 1000, "bf16"), (333, 136, 2048, "bf16"), (700, 2048, 1024, "f16"),
    (1025, 264, 2104, "bf16"),
]


def ffn_inputs(m, d, f, dt, ints=False, seed=0):
    g = np.random.default_rng([seed, m, d, f])
    if ints:
        return [gpu(v, dt) for v in (g.integers(-2, 3, (m, d)), g.integers(-1, 2, (d, 2 * f)), g.integers(-2, 3, (m, f)))]
    return [gpu(v, dt) for v in (g.standard_normal((m, d)), g.standard_normal((d, 2 * f)) / np.sqrt(d),
                                 g.standard_normal((m, f)))]


@pytest.mark.parametrize("m,d,f,dt", FFN)
def test_gated_ffn_of_whole_numbers(m, d, f, dt):
    """Small whole numbers: the saved projections are exact."""
    log(f"gated ffn {m} x {d} x {f} {dt}")
    (x, xv), (w, wv), _ = ffn_inputs(m, d, f, dt, ints=True)
    gate_up, keep = guarded((m, 2 * f), x.dtype)
    h, keep_h = guarded((m, f), x.dtype)
    tgc.gated_ffn(x, w, h=h, gate_up=gate_up)
    torch.cuda.synchronize()
    keep("gate_up")
    keep_h("h")
    same_bits(gate_up, xv @ wv, dt, "gate_up")
    equal(h, tgc.gated_ffn(x, w)[0], "h without saving")


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("m,d,f,dt", FFN)
def test_gated_ffn(m, d, f, dt, kind):
    log(f"gated ffn {m} x {d} x {f} {dt} {kind}")
    (x, xv), (w, wv), _ = ffn_inputs(m, d, f, dt)
    h, both = tgc.gated_ffn(x, w, act=kind, save=True)
    for a, b in zip((h, both), tgc.gated_ffn(x, w, act=kind, save=True)):
        equal(a, b, "twice")
    ref, rb = B.gated_ffn(xv, wv, kind)
    off = (2 * (d + 8) + 4) * U * (np.abs(xv) @ np.abs(wv))
    within(both, rb, off * (1 + HALF[dt]) + HALF[dt] * np.abs(rb) + TINY[dt], "gate_up")
    # |act'| <= 1.13
    g, u = rb[:, :f], rb[:, f:]
    own = act_bounds(rb, kind)[0] + 1.13 * off[:, :f] * (np.abs(u) + off[:, f:]) + np.abs(B.act(g, kind)[0]) * off[:, f:]
    within(h, ref, own * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], "h")


@pytest.mark.parametrize("m,d,f,dt", FFN)
def test_gated_ffn_backward(m, d, f, dt):
    log(f"gated ffn backward {m} x {d} x {f} {dt}")
    (x, xv), (w, wv), (dh, dhv) = ffn_inputs(m, d, f, dt)
    gate_up, gv = gpu(np.random.default_rng(m).standard_normal((m, 2 * f)), dt)
    dx, keep = guarded((m, d), x.dtype)
    dw, keep_w = guarded((d, 2 * f), x.dtype)
    tgc.gated_ffn_backward(dh, x, w, gate_up, dx=dx, dw=dw)
    torch.cuda.synchronize()
    keep("dx")
    keep_w("dw")
    for a, b in zip((dx, dw), tgc.gated_ffn_backward(dh, x, w, gate_up)):
        equal(a, b, "twice")
    only = tgc.gated_ffn_backward(dh, x, w, gate_up, need_dw=False)
    equal(only[0], dx, "dx alone")
    assert only[1] is None
    only = tgc.gated_ffn_backward(dh, x, w, gate_up, need_dx=False)
    equal(only[1], dw, "dw alone")
    # the projections' gradient as the operator rounds it, then the two products
    dgu = tgc.gated_act_backward(dh, gate_up).double().cpu().numpy()
    for got, a, b, terms, what in ((dx, dgu, wv.T, 2 * f, "dx"), (dw, xv.T, dgu, m, "dw")):
        ref = a @ b
        off = (2 * (terms + 8) + 4) * U * (np.abs(a) @ np.abs(b))
        within(got, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], what)
    # and against the formula, the projections' gradient rounded once more
    rx, rw = B.gated_ffn_backward(dhv, xv, wv, gv, "silu")
    dv = np.abs(B.gated_act_backward(dhv, gv, "silu"))
    for got, ref, size, terms, what in ((dx, rx, dv @ np.abs(wv.T), 2 * f, "dx"), (dw, rw, np.abs(xv.T) @ dv, m, "dw")):
        off = (HALF[dt] * 1.01 + (2 * (terms + 8) + 200) * U) * size + 2 * TINY[dt] * terms
        within(got, ref, off * (1 + HALF[dt]) + HALF[dt] * np.abs(ref) + TINY[dt], what + " by the formula")


@pytest.mark.parametrize("m,d,f,dt", [(40, 264, 136, "bf16"), (300, 1040, 1000, "f16")])
def test_gated_ffn_backward_computes_the_projections_again(m, d, f, dt):
    (x, _), (w, _), (dh, _) = ffn_inputs(m, d, f, dt)
    _, gate_up = tgc.gated_ffn(x, w, act="gelu", save=True)
    for a, b in zip(tgc.gated_ffn_backward(dh, x, w, act="gelu"), tgc.gated_ffn_backward(dh, x, w, gate_up, act="gelu")):
        equal(a, b, "recomputed")


def test_gated_ffn_without_rows():
    x, w = torch.empty(0, 64, device="cuda").bfloat16(), torch.ones(64, 32, device="cuda").bfloat16()
    assert tgc.gated_ffn(x, w)[0].shape == (0, 16)
    dx, dw = tgc.gated_ffn_backward(torch.empty(0, 16, device="cuda").bfloat16(), x, w, dw=torch.ones_like(w))
    assert dx.shape == (0, 64) and not dw.any()


def test_gated_ffn_keeps_bad_values_in_their_rows_and_columns():
    for m in (3, 40, 200):
        (x, _), (w, _), _ = ffn_inputs(m, 520, 264, "bf16")
        want = tgc.gated_ffn(x, w)[0]
        x2, w2 = x.clone(), w.clone()
        x2[1, 519] = float("nan")
        w2[519, 263] = float("nan")      # the last gate column
        w2[0, 264 + 8] = float("nan")    # an up column
        got = tgc.gated_ffn(x2, w2)[0]
        assert torch.isnan(got[1]).all() and torch.isnan(got[:, 263]).all() and torch.isnan(got[:, 8]).all()
        rows = [i for i in range(m) if i != 1]
        cols = [i for i in range(264) if i not in (8, 263)]
        equal(got[rows][:, cols], want[rows][:, cols], "the others")


# ------------------------------------------------------------------ streams and graphs
def block_state(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, d, f = 150, 528, 272
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return {"x": n(t, d), "res": n(t, d), "gamma": n(d), "w": n(d, 2 * f) / 16, "wn": n(2 * f, d) / 16, "dh": n(t, f)}


def whole_pass(s):
    """Every operator once."""
    y, rstd, total = tgc.rms_norm(s["x"], s["gamma"], residual=s["res"])
    h, both = tgc.gated_ffn(y, s["w"], save=True)
    dy, dw = tgc.gated_ffn_backward(s["dh"], y, s["w"], both)
    dx, dgamma = tgc.rms_norm_backward(dy, total, s["gamma"], rstd, dsum=s["res"])
    one = tgc.gated_ffn(y[:1], s["w"], act="gelu")[0]
    again = tgc.gated_ffn_backward(s["dh"], y, s["w"])
    q, qs, _ = tgc.rms_norm_fp8(s["x"], s["gamma"])
    w8, ws = tgc.quantize_fp8(s["wn"], block_rows=128)
    p = tgc.matmul_fp8(q, qs, w8, ws)
    p1 = tgc.matmul_fp8(q[:1], qs[:, :1].contiguous(), w8, ws, dtype=torch.float32)
    a, as_ = tgc.gated_act_fp8(p)
    return [y, rstd, total, h, both, dy, dw, dx, dgamma, one, *again, q, qs, w8, ws, p, p1, a, as_, tgc.gated_act(p),
            tgc.gated_act_backward(s["dh"], p)]


def test_the_block_in_one_graph():
    """A graph that holds every operator, replayed on changing inputs with eager
    calls between the replays: each replay gives the eager bits."""
    states = [block_state(i) for i in range(3)]
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
    s = block_state(5)
    want = tgc.gated_ffn_backward(s["dh"], s["x"], s["w"])
    want_norm = tgc.rms_norm_backward(s["x"], s["res"], s["gamma"], torch.ones(150, device="cuda"))
    rstd = torch.ones(150, device="cuda")
    q, qs = tgc.quantize_fp8(s["x"])
    w8, ws = tgc.quantize_fp8(s["wn"], block_rows=128)
    want_p = tgc.matmul_fp8(q, qs, w8, ws)
    torch.cuda.synchronize()
    for _ in range(4):
        got = tgc.gated_ffn_backward(s["dh"], s["x"], s["w"], stream=side)
        norm = tgc.rms_norm_backward(s["x"], s["res"], s["gamma"], rstd, stream=side)
        p = tgc.matmul_fp8(q, qs, w8, ws, stream=side)
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]   # takes freed memory of this stream
        side.synchronize()
        for a, b in zip((*got, *norm, p), (*want, *want_norm, want_p)):
            equal(a, b, "on another stream")
        del junk


# ------------------------------------------------------------------ with the fused matmuls
def test_the_block_around_the_collective_matmuls():
    """The gate/up product by the all-gather matmul, the activation, the down
    product by the reduce-scatter: the tensor-parallel form of the block, whose
    projections are bit for bit those that gated_ffn saves."""
    world, rank, m, d, f = 2, 0, 256, 512, 256
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    shards, w, down = [n(m // world, d) for _ in range(world)], n(d, 2 * f) / 16, n(f, d) / 16
    gamma = n(d)
    normed = [tgc.rms_norm(s, gamma)[0] for s in shards]
    both, gathered = tgc.allgather_matmul(normed[rank], [None, normed[1]], w, rank, split=2, v2=True)
    h = tgc.gated_act(both)
    part = n(m, d)
    y, partial = tgc.matmul_reduce_scatter(h, down, [None, part], rank, split=2)
    torch.cuda.synchronize()
    fused, saved = tgc.gated_ffn(gathered, w, save=True)
    hv = h.double().cpu().numpy()
    ref = B.gated_act(both.double().cpu().numpy(), "silu")
    off, _ = act_bounds(both.double().cpu().numpy(), "silu")
    within(h, ref, off * 1.01 + HALF["bf16"] * np.abs(ref) + TINY["bf16"], "h")
    # the two products may round differently where their sums' order differs
    size = np.abs(gathered.double().cpu().numpy()) @ np.abs(w.double().cpu().numpy())
    exact = gathered.double().cpu().numpy() @ w.double().cpu().numpy()
    bound = 2 * (d + 8) * U * size * 1.01 + HALF["bf16"] * np.abs(exact)
    within(saved, exact, bound, "saved projections")
    within(both, exact, bound, "the all-gather matmul's")
    want = (hv @ down.double().cpu().numpy())
    within(partial, want, 2 * (f + 8) * U * (np.abs(hv) @ np.abs(down.double().cpu().numpy())) * 1.01 +
           HALF["bf16"] * np.abs(want), "down")
