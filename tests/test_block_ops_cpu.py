"""Refusals of the gated feed-forward block's operators, on the host: the C entry
points with placeholder addresses (nothing may be enqueued, so these run only
where no GPU is visible), and the binding's checks of tensors."""
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tensor_gemm_collective_amd import coc

no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers: host-only environment")

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS = 1, 3, 5, 6, 7, 9
G = 1 << 34   # placeholder addresses, 16 GiB apart


def at(i):
    return G * (i + 1)


def entry(name, pointers, sizes, after=(), ws=False):
    """A call of coc_<name> with placeholder pointers, then the sizes and other values."""
    def call(**kw):
        a = {k: at(i) for i, k in enumerate(pointers)} | dict(sizes) | dict(after) | dict(ws=at(20), nws=1 << 40) | kw
        values = [a[k] for k in pointers] + [a[k] for k, _ in (*sizes, *after)] + ([a["ws"], a["nws"]] if ws else [])
        return getattr(tgc.lib(), "coc_" + name)(*values, None)
    call.__name__ = name
    return call


NORM = (("rows", 4), ("n", 64))
ACT = (("rows", 4), ("f", 64), ("act", 0), ("dt", 2))
FFN = (("m", 4), ("d", 64), ("f", 32), ("act", 0), ("dt", 2))
RMS = ["x", "residual", "gamma", "y", "sum_out", "rstd"]
RMS8 = ["x", "residual", "gamma", "q", "scales", "sum_out", "rstd"]
RMSB = ["dy", "x", "gamma", "rstd", "dsum", "dx", "dgamma"]
rms = entry("rms_norm", RMS, NORM, (("eps", 1e-5), ("dt", 2), ("pdt", 2)))
rms8 = entry("rms_norm_fp8", RMS8, NORM, (("eps", 1e-5), ("dt", 2), ("pdt", 2)))
rmsb = entry("rms_norm_backward", RMSB, NORM, (("dt", 2), ("pdt", 0)), ws=True)
quant = entry("quantize_fp8", ["x", "q", "scales"], NORM, (("block_rows", 1), ("dt", 2)))
mm8 = entry("matmul_fp8", ["x", "xs", "w", "wsc", "y"], (("m", 4), ("n", 24), ("k", 272)), (("dt", 2),), ws=True)
gact = entry("gated_act", ["gate_up", "h"], ACT)
gact8 = entry("gated_act_fp8", ["gate_up", "q", "scales"], ACT)
gactb = entry("gated_act_backward", ["dh", "gate_up", "dgate_up"], ACT)
ffn = entry("gated_ffn", ["x", "w", "h", "gate_up"], FFN, ws=True)
ffnb = entry("gated_ffn_backward", ["dh", "x", "w", "gate_up", "dx", "dw"], FFN, ws=True)

CASES = [
    *[(rms, {k: None}, NULL) for k in RMS if k != "residual"],
    *[(rms8, {k: None}, NULL) for k in RMS8 if k != "residual"],
    *[(rmsb, {k: None}, NULL) for k in RMSB if k != "dsum"],
    *[(f, kw, s) for f in (rms, rms8) for kw, s in (
        (dict(rows=-1), SHAPE), (dict(n=0), SHAPE), (dict(n=32784), SHAPE), (dict(rows=1 << 25), SHAPE),
        (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(dt=3), DTYPE), (dict(dt=2, pdt=1), DTYPE),
        (dict(x=at(0) + 1), ALIGN), (dict(rstd=at(6) + 2), ALIGN), (dict(sum_out=at(1)), ALIAS),
        (dict(sum_out=at(0) + 510), ALIAS))],
    (rms, dict(y=at(0)), ALIAS), (rms8, dict(q=at(3) + 8), ALIGN), (rms8, dict(scales=at(4) + 2), ALIGN),
    (rms8, dict(q=at(0)), ALIAS), (rms8, dict(scales=at(3) + 64), ALIAS), (rms8, dict(n=72), SHAPE),
    (rms8, dict(rstd=at(4) + 12), ALIAS),
    (rmsb, dict(rows=100, ws=None), WORKSPACE), (rmsb, dict(rows=100, nws=8), WORKSPACE),
    (rmsb, dict(rows=100, ws=at(20) + 2), ALIGN), (rmsb, dict(dx=at(0)), ALIAS), (rmsb, dict(rows=100, ws=at(5)), ALIAS), (rmsb, dict(pdt=1), DTYPE), (rmsb, dict(n=32769), SHAPE),
    (rmsb, dict(rows=0, dgamma=None), NULL),
    *[(quant, {k: None}, NULL) for k in ("x", "q", "scales")],
    (quant, dict(n=72), SHAPE), (quant, dict(rows=-1), SHAPE), (quant, dict(block_rows=2), DTYPE),
    (quant, dict(block_rows=0), DTYPE), (quant, dict(dt=3), DTYPE), (quant, dict(q=at(1) + 4), ALIGN),
    (quant, dict(q=at(0) + 496), ALIAS), (quant, dict(scales=at(1)), ALIAS), (quant, dict(rows=1 << 25), SHAPE),
    *[(mm8, {k: None}, NULL) for k in ("x", "xs", "w", "wsc", "y")],
    (mm8, dict(k=264), SHAPE), (mm8, dict(m=-1), SHAPE), (mm8, dict(n=-1), SHAPE), (mm8, dict(k=-16), SHAPE),
    (mm8, dict(dt=3), DTYPE), (mm8, dict(x=at(0) + 8), ALIGN), (mm8, dict(w=at(2) + 4), ALIGN),
    (mm8, dict(xs=at(1) + 2), ALIGN), (mm8, dict(y=at(4) + 1), ALIGN), (mm8, dict(y=at(0) + 1000), ALIAS),
    (mm8, dict(y=at(3)), ALIAS), (mm8, dict(m=40, k=8192, ws=None), WORKSPACE),
    (mm8, dict(m=40, k=8192, nws=64), WORKSPACE), (mm8, dict(m=40, k=8192, ws=at(20) + 4), ALIGN),
    (mm8, dict(m=40, k=8192, ws=at(4)), ALIAS), (mm8, dict(m=1 << 20, n=1 << 20), SHAPE),
    *[(gact, {k: None}, NULL) for k in ("gate_up", "h")], *[(gact8, {k: None}, NULL) for k in ("gate_up", "q", "scales")],
    *[(gactb, {k: None}, NULL) for k in ("dh", "gate_up", "dgate_up")],
    *[(f, kw, s) for f in (gact, gact8, gactb) for kw, s in (
        (dict(act=2), DTYPE), (dict(act=-1), DTYPE), (dict(dt=5), DTYPE), (dict(f=0), SHAPE), (dict(rows=-1), SHAPE),
        (dict(f=1 << 30), SHAPE), (dict(rows=1 << 25), SHAPE), (dict(gate_up=at(1) + 1), ALIGN))],
    (gact, dict(h=at(0) + 4), ALIAS), (gact8, dict(f=72), SHAPE), (gact8, dict(q=at(1) + 8), ALIGN),
    (gactb, dict(dgate_up=at(1)), ALIAS), (gactb, dict(dgate_up=at(0)), ALIAS),
    *[(ffn, {k: None}, NULL) for k in ("x", "w", "h")], *[(ffnb, {k: None}, NULL) for k in ("dh", "x", "w")],
    *[(f, kw, s) for f in (ffn, ffnb) for kw, s in (
        (dict(dt=0), DTYPE), (dict(act=2), DTYPE), (dict(d=60), SHAPE), (dict(f=12), SHAPE), (dict(d=0), SHAPE),
        (dict(f=0), SHAPE), (dict(m=-1), SHAPE), (dict(d=1 << 16, f=1 << 15), SHAPE), (dict(f=1 << 31), SHAPE),
        (dict(x=at(1) + 8), ALIGN), (dict(gate_up=at(3) + 2), ALIGN), (dict(d=8192, ws=None), WORKSPACE),
        (dict(d=8192, nws=64), WORKSPACE), (dict(d=8192, ws=at(20) + 8), ALIGN), (dict(d=8192, ws=at(3)), ALIAS))],
    (ffn, dict(h=at(1)), ALIAS), (ffn, dict(gate_up=at(2) + 240), ALIAS), (ffnb, dict(dx=at(1)), ALIAS),
    (ffnb, dict(dw=at(2)), ALIAS), (ffnb, dict(dw=at(4)), ALIAS),
]


@no_gpu_only
@pytest.mark.parametrize("fn,kw,status", CASES, ids=lambda v: getattr(v, "__name__", str(v)))
def test_entry_points_refuse(fn, kw, status):
    assert coc.STATUS[fn(**kw)] == coc.STATUS[status]
    assert tgc.lib().coc_last_error().decode() != ""


@no_gpu_only
def test_calls_without_rows_do_nothing():
    assert rms(rows=0, x=None, y=None) == 0 and rms8(rows=0, x=None, q=None) == 0
    assert quant(rows=0, x=None) == 0 and quant(n=0, x=None) == 0
    assert mm8(m=0, x=None, y=None, ws=None) == 0 and mm8(n=0, w=None, y=None, ws=None) == 0
    assert gact(rows=0, h=None) == 0 and gact8(rows=0, q=None) == 0 and gactb(rows=0, dh=None) == 0
    assert ffn(m=0, x=None, h=None, ws=None) == 0
    assert ffnb(m=0, dh=None, x=None, dw=None, ws=None) == 0
    assert ffnb(dx=None, dw=None) == 0


def test_workspace_sizes():
    L = tgc.lib()
    assert L.coc_rms_norm_backward_workspace_bytes(0, 64) == 0
    assert L.coc_rms_norm_backward_workspace_bytes(3, 64) == 0          # one workgroup
    assert L.coc_rms_norm_backward_workspace_bytes(300, 64) >= 2 * 64 * 4
    assert L.coc_rms_norm_backward_workspace_bytes(3, 32769) == 0
    assert L.coc_matmul_fp8_workspace_bytes(0, 8, 16) == 0 and L.coc_matmul_fp8_workspace_bytes(8, 8, 8) == 0
    assert L.coc_gated_ffn_workspace_bytes(4, 60, 64) == 0
    # one token's sums are split over the GPU
    assert L.coc_gated_ffn_workspace_bytes(1, 8192, 3584) >= 2 * 3584 * 4 * 2
    assert L.coc_gated_ffn_backward_workspace_bytes(100, 64, 32) >= 100 * 64 * 2


def _f(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


F8, F32 = torch.float8_e4m3fn, torch.float32


@pytest.mark.parametrize("call,error", [
    (lambda: tgc.rms_norm(_f(4, 8), _f(8)), ValueError),                                      # not on the GPU
    (lambda: tgc.rms_norm(_f(4, 8), _f(7)), ValueError),
    (lambda: tgc.rms_norm(_f(8), _f(8)), ValueError),
    (lambda: tgc.rms_norm(_f(8, 4).t(), _f(8)), ValueError),                                  # not dense
    (lambda: tgc.rms_norm(_f(4, 8, dtype=torch.float64), _f(8)), TypeError),
    (lambda: tgc.rms_norm(_f(4, 8), _f(8), residual=_f(4, 8, dtype=F32)), TypeError),
    (lambda: tgc.rms_norm_fp8(_f(4, 16), _f(16)), ValueError),
    (lambda: tgc.rms_norm_fp8(_f(4, 16), _f(16), q=_f(4, 16)), TypeError),
    (lambda: tgc.rms_norm_fp8(_f(4, 16), _f(16), q=_f(4, 16, dtype=F8), scales=_f(4, 1, dtype=F32)), ValueError),
    (lambda: tgc.rms_norm_backward(_f(4, 8), _f(4, 8), _f(8), _f(4)), TypeError),             # statistic not fp32
    (lambda: tgc.rms_norm_backward(_f(4, 9), _f(4, 8), _f(8), _f(4, dtype=F32)), ValueError),
    (lambda: tgc.quantize_fp8(_f(4, 16)), ValueError),
    (lambda: tgc.quantize_fp8(_f(4, 16, dtype=torch.int8)), TypeError),
    (lambda: tgc.matmul_fp8(_f(4, 16), _f(1, 4, dtype=F32), _f(8, 16, dtype=F8), _f(1, 1, dtype=F32)), TypeError),
    (lambda: tgc.matmul_fp8(_f(4, 16, dtype=F8), _f(4, 1, dtype=F32), _f(8, 16, dtype=F8), _f(1, 1, dtype=F32)), ValueError),
    (lambda: tgc.matmul_fp8(_f(4, 16, dtype=F8), _f(1, 4, dtype=F32), _f(8, 32, dtype=F8), _f(1, 1, dtype=F32)), ValueError),
    (lambda: tgc.matmul_fp8(_f(4, 16, dtype=F8), _f(1, 4, dtype=F32), _f(8, 16, dtype=F8), _f(1, 1)), TypeError),
    (lambda: tgc.matmul_fp8(_f(4, 16, dtype=F8), _f(1, 4, dtype=F32), _f(8, 16, dtype=F8), _f(1, 1, dtype=F32)), ValueError),
    (lambda: tgc.gated_act(_f(4, 7)), ValueError),                                            # odd
    (lambda: tgc.gated_act(_f(4, 8), act="relu"), ValueError),
    (lambda: tgc.gated_act(_f(4, 8)), ValueError),
    (lambda: tgc.gated_act_fp8(_f(4, 32)), ValueError),
    (lambda: tgc.gated_act_backward(_f(4, 8), _f(4, 8)), ValueError),
    (lambda: tgc.gated_act_backward(_f(4, 4, dtype=F32), _f(4, 8)), TypeError),
    (lambda: tgc.gated_ffn(_f(4, 8), _f(8, 32)), ValueError),
    (lambda: tgc.gated_ffn(_f(4, 8), _f(16, 32)), ValueError),
    (lambda: tgc.gated_ffn(_f(4, 8), _f(8, 32, dtype=torch.float16)), TypeError),
    (lambda: tgc.gated_ffn(_f(4, 8), _f(8, 31)), ValueError),
    (lambda: tgc.gated_ffn_backward(_f(4, 16), _f(4, 8), _f(8, 32), _f(4, 16)), ValueError),
    (lambda: tgc.gated_ffn_backward(_f(4, 15), _f(4, 8), _f(8, 32)), ValueError),
])
def test_binding_refuses(call, error):
    with pytest.raises(error):
        call()
