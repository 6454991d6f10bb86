"""Cases and plain forms of the gated feed-forward block's operators, in 16 bits for training and in 8 for serving.

One tensor-parallel rank's share of a block: the root-mean-square norm in front
of it (with the residual's addition, its backward pass, and an output in 8 bits
with a scale for each 128 of a row), the gated projections with their
activation and backward pass, and the matrix product in 8-bit floating point
with a scale for each block of 128 that serving runs them on, with the
quantisation of its operands.

A case is a dict whose "op" names the operator; `prepare` makes what a
program holds before the call, `run` makes one pass.  With `own` false `run`
computes the plain form in elementary torch operations; with `own` true it
calls the library.  `exact` is the operators' definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 128           # values along a row that share a scale
TOP = 448.0           # the largest e4m3 value
LEAST = 2.0 ** -96    # blocks below this are scaled as if this were their largest value
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token's norm in decoding, straight into the 8 bits of the next product
        {"name": "rms_fp8_token", "op": "rms_norm_fp8", "rows": 1, "n": 8192, "dtype": "bf16", "residual": True},
        # a prompt's, with the residual's addition
        {"name": "rms_fp8_prompt", "op": "rms_norm_fp8", "rows": 4096, "n": 8192, "dtype": "bf16", "residual": True},
        # the training norm's backward pass, the residual's gradient joined in
        {"name": "rms_backward", "op": "rms_norm_backward", "rows": 2048, "n": 8192, "dtype": "bf16",
         "residual": True},
        # a gate/up weight shard brought into 8 bits, a scale for each 128 x 128
        {"name": "quantize_weight", "op": "quantize_fp8", "rows": 7168, "n": 8192, "dtype": "bf16",
         "block_rows": 128},
        # activations that no norm made: a ragged batch in 32 bits, a scale for each 128 of a row
        {"name": "quantize_rows", "op": "quantize_fp8", "rows": 1001, "n": 1040, "dtype": "f32", "block_rows": 1},
        # one token through the gate/up product in 8 bits
        {"name": "fp8_token", "op": "matmul_fp8", "m": 1, "n": 7168, "k": 8192, "dtype": "bf16"},
        # a short ragged batch through a product with no round size
        {"name": "fp8_ragged", "op": "matmul_fp8", "m": 333, "n": 1999, "k": 1040, "dtype": "f16"},
        # a prompt through it
        {"name": "fp8_prompt", "op": "matmul_fp8", "m": 4096, "n": 7168, "k": 8192, "dtype": "bf16"},
        # one token through both projections, the activation and the product
        {"name": "gated_token", "op": "gated_ffn", "m": 1, "d": 8192, "f": 3584, "dtype": "bf16", "act": "silu",
         "save": False},
        # a training step's forward pass, which keeps the projections for the backward pass
        {"name": "gated_train", "op": "gated_ffn", "m": 4096, "d": 8192, "f": 3584, "dtype": "bf16", "act": "silu",
         "save": True},
        # its backward pass down to the input and the weights
        {"name": "gated_backward", "op": "gated_ffn_backward", "m": 4096, "d": 8192, "f": 3584, "dtype": "bf16",
         "act": "silu"},
        # the activation and the product behind an 8-bit gate/up product, into the 8 bits of the down product
        {"name": "act_fp8", "op": "gated_act_fp8", "m": 4096, "f": 3584, "dtype": "bf16", "act": "silu"},
    ]


def draw(rng):
    def spread(lo, hi, odd=0.3):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return v | 1 if rng.random() < odd and v < hi else v

    def eights(lo, hi, of=8):
        return of * spread(lo // of, hi // of)

    op = rng.choice(["rms_norm", "rms_norm_fp8", "rms_norm_backward", "quantize_fp8", "matmul_fp8", "matmul_fp8",
                     "gated_ffn", "gated_ffn", "gated_ffn_backward", "gated_act", "gated_act_fp8",
                     "gated_act_backward"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    act = rng.choice(["silu", "gelu"])
    if op.startswith("rms_norm"):
        n = eights(64, 14336, 16) if op == "rms_norm_fp8" else spread(64, 14336)
        rows = spread(1, max(2, min(16384, 2048 * 8192 // n)))
        return {"op": op, "rows": rows, "n": n, "dtype": dtype, "residual": rng.random() < 0.5}
    if op == "quantize_fp8":
        n = eights(64, 14336, 16)
        rows = spread(1, max(2, min(16384, 3584 * 8192 // n)))
        return {"op": op, "rows": rows, "n": n, "dtype": dtype, "block_rows": rng.choice([1, 128])}
    if op == "matmul_fp8":
        return {"op": op, "m": spread(1, 4096), "n": spread(16, 7168), "k": eights(64, 8192, 16), "dtype": dtype}
    if op.startswith("gated_ffn"):
        case = {"op": op, "m": spread(1, 4096), "d": eights(64, 8192), "f": eights(64, 3584),
                "dtype": rng.choice(["bf16", "f16"]), "act": act}
        if op == "gated_ffn":
            case["save"] = rng.random() < 0.5
        return case
    f = eights(64, 8192, 16) if op == "gated_act_fp8" else spread(64, 8192)
    return {"op": op, "m": spread(1, max(2, min(16384, 1792 * 4096 // f))), "f": f, "dtype": dtype, "act": act}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype, sigma=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(dtype)


def _hidden(gen, rows, n, dtype):
    """Activations of which a few channels are much larger than the others, as behind a norm."""
    channel = 1.0 + 6.0 * (torch.rand(n, generator=gen, device="cuda") < 0.01).float()
    return (torch.randn(rows, n, generator=gen, device="cuda") * channel).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    if op.startswith("rms_norm"):
        rows, n = case["rows"], case["n"]
        s["x"] = _hidden(gen, rows, n, dt)
        s["gamma"] = _normal(gen, (n,), dt, 0.1) + 1.0
        s["other"] = _normal(gen, (rows, n), dt) if case["residual"] else None
        if op == "rms_norm_backward":
            s["dy"] = _normal(gen, (rows, n), dt)
            s["rstd"] = s["x"].float().square().mean(1).add(EPS).rsqrt()
    elif op == "quantize_fp8":
        s["x"] = _hidden(gen, case["rows"], case["n"], dt)
    elif op == "matmul_fp8":
        m, n, k = case["m"], case["n"], case["k"]
        s["x"], s["xs"] = _quantize(_hidden(gen, m, k, torch.float32), 1)
        s["w"], s["ws"] = _quantize(_normal(gen, (n, k), torch.float32, k ** -0.5), BLOCK)
    elif op.startswith("gated_ffn"):
        m, d, f = case["m"], case["d"], case["f"]
        s["x"] = _normal(gen, (m, d), dt)
        s["w"] = _normal(gen, (d, 2 * f), dt, d ** -0.5)   # gate columns, then up columns
        if op == "gated_ffn_backward":
            s["gate_up"] = _normal(gen, (m, 2 * f), dt)
            s["dh"] = _normal(gen, (m, f), dt)
    else:
        s["gate_up"] = _normal(gen, (case["m"], 2 * case["f"]), dt)
        if op == "gated_act_backward":
            s["dh"] = _normal(gen, (case["m"], case["f"]), dt)
    return s


# ------------------------------------------------------------------ plain forms
def _blocks(y, block_rows):
    """y (rows x n) with zeros up to whole blocks, as (row blocks, block_rows, column blocks, 128)."""
    rows, n = y.shape
    full = y.new_zeros(-(-rows // block_rows) * block_rows, -(-n // BLOCK) * BLOCK)
    full[:rows, :n] = y
    return full.view(-1, block_rows, full.shape[1] // BLOCK, BLOCK)


def _quantize(y, block_rows):
    """e4m3 values and scales of y (32 bits).  A row's scales: (column blocks, rows); those of
    128 x 128 blocks: (row blocks, column blocks)."""
    rows, n = y.shape
    b = _blocks(y, block_rows)
    top = b.abs().amax((1, 3)).clamp(min=LEAST)
    q = (b * (TOP / top)[:, None, :, None]).reshape(-1, b.shape[2] * BLOCK)[:rows, :n]
    scales = top / TOP
    return q.to(torch.float8_e4m3fn), (scales.t() if block_rows == 1 else scales).contiguous()


def _wide(q, scales, block_rows):
    """What e4m3 values and their scales stand for, in 32 bits."""
    rows, n = q.shape
    s = scales.t() if block_rows == 1 else scales.repeat_interleave(BLOCK, 0)[:rows]
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :n]


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _slope(g, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return p * (1.0 + g * (1.0 - p))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _act_backward(s):
    f = s["f"]
    g, u, dh = s["gate_up"][:, :f].float(), s["gate_up"][:, f:].float(), s["dh"].float()
    return torch.cat([dh * u * _slope(g, s["act"]), dh * _act(g, s["act"])], 1)


def _plain(s):
    op = s["op"]
    if op in ("rms_norm", "rms_norm_fp8"):
        x = s["x"]
        if s["residual"]:
            x = (x.float() + s["other"].float()).to(x.dtype)
        h = x.float()
        rstd = 1.0 / torch.sqrt(h.square().mean(1) + EPS)
        y = h * rstd[:, None] * s["gamma"].float()
        out = {"rstd": rstd, "sum": x if s["residual"] else None}
        if op == "rms_norm":
            out["y"] = y.to(x.dtype)
        else:
            out["q"], out["scales"] = _quantize(y, 1)
        return out
    if op == "rms_norm_backward":
        dy = s["dy"].float()
        xhat = s["x"].float() * s["rstd"][:, None]
        g = dy * s["gamma"].float()
        dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if s["residual"]:
            dx = dx + s["other"].float()
        return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0).to(s["gamma"].dtype)}
    if op == "quantize_fp8":
        q, scales = _quantize(s["x"].float(), s["block_rows"])
        return {"q": q, "scales": scales}
    if op == "matmul_fp8":
        return (_wide(s["x"], s["xs"], 1) @ _wide(s["w"], s["ws"], BLOCK).t()).to(DTYPES[s["dtype"]])
    f, dt = s["f"], DTYPES[s["dtype"]]
    if op == "gated_ffn":
        both = s["x"].float() @ s["w"].float()
        h = (_act(both[:, :f], s["act"]) * both[:, f:]).to(dt)
        return {"h": h, "gate_up": both.to(dt) if s["save"] else None}
    if op == "gated_ffn_backward":
        d = _act_backward(s)
        return {"dx": (d @ s["w"].float().t()).to(dt), "dw": (s["x"].float().t() @ d).to(dt)}
    if op == "gated_act_backward":
        return _act_backward(s).to(dt)
    h = _act(s["gate_up"][:, :f].float(), s["act"]) * s["gate_up"][:, f:].float()
    if op == "gated_act":
        return h.to(dt)
    q, scales = _quantize(h, 1)
    return {"q": q, "scales": scales}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import tensor_gemm_collective_amd as tgc
    op = s["op"]
    if op == "rms_norm":
        got = tgc.rms_norm(s["x"], s["gamma"], residual=s["other"], eps=EPS)
        return {"y": got[0], "rstd": got[1], "sum": got[2] if s["residual"] else None}
    if op == "rms_norm_fp8":
        got = tgc.rms_norm_fp8(s["x"], s["gamma"], residual=s["other"], eps=EPS)
        return {"q": got[0], "scales": got[1], "rstd": got[2], "sum": got[3] if s["residual"] else None}
    if op == "rms_norm_backward":
        dx, dgamma = tgc.rms_norm_backward(s["dy"], s["x"], s["gamma"], s["rstd"], dsum=s["other"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "quantize_fp8":
        q, scales = tgc.quantize_fp8(s["x"], block_rows=s["block_rows"])
        return {"q": q, "scales": scales}
    if op == "matmul_fp8":
        return tgc.matmul_fp8(s["x"], s["xs"], s["w"], s["ws"], dtype=DTYPES[s["dtype"]])
    if op == "gated_ffn":
        h, gate_up = tgc.gated_ffn(s["x"], s["w"], act=s["act"], save=s["save"])
        return {"h": h, "gate_up": gate_up}
    if op == "gated_ffn_backward":
        dx, dw = tgc.gated_ffn_backward(s["dh"], s["x"], s["w"], s["gate_up"], act=s["act"])
        return {"dx": dx, "dw": dw}
    if op == "gated_act_backward":
        return tgc.gated_act_backward(s["dh"], s["gate_up"], act=s["act"])
    if op == "gated_act":
        return tgc.gated_act(s["gate_up"], act=s["act"])
    q, scales = tgc.gated_act_fp8(s["gate_up"], act=s["act"])
    return {"q": q, "scales": scales}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, es = case["op"], 4 if case["dtype"] == "f32" else 2
    if op.startswith("rms_norm") or op == "quantize_fp8":
        rows, n = case["rows"], case["n"]
        cells, scales = rows * n, 4 * rows * -(-n // BLOCK)
        if op == "quantize_fp8":
            return {"bytes": cells * (es + 1) + scales // case["block_rows"], "flops": 3 * cells}
        if op == "rms_norm_backward":
            return {"bytes": es * (cells * (4 if case["residual"] else 3) + 2 * n) + 4 * rows, "flops": 12 * cells}
        out = cells + scales if op == "rms_norm_fp8" else es * cells
        return {"bytes": es * (cells * (3 if case["residual"] else 1) + n) + out + 4 * rows, "flops": 7 * cells}
    if op == "matmul_fp8":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        return {"bytes": m * k + n * k + es * m * n + 4 * kb * (m + -(-n // BLOCK)), "flops": 2 * m * n * k}
    m, f = case["m"], case["f"]
    if op.startswith("gated_ffn"):
        d = case["d"]
        if op == "gated_ffn":
            return {"bytes": es * (m * d + 2 * d * f + m * f * (3 if case["save"] else 1)),
                    "flops": 4 * m * d * f + 6 * m * f}
        return {"bytes": es * (2 * m * d + 4 * d * f + 3 * m * f), "flops": 8 * m * d * f + 12 * m * f}
    if op == "gated_act_fp8":
        return {"bytes": 2 * es * m * f + m * f + 4 * m * -(-f // BLOCK), "flops": 9 * m * f}
    return {"bytes": es * m * f * (3 if op == "gated_act" else 5), "flops": (6 if op == "gated_act" else 12) * m * f}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_scaled(y, block_rows):
    """y over its scale (not rounded to 8 bits), and the scales, column block by column block."""
    rows, n = y.shape
    over, scales = torch.empty_like(y), []
    first = torch.arange(rows, device="cuda") // block_rows
    for c in range(0, n, BLOCK):
        part = y[:, c:c + BLOCK]
        top = torch.zeros(int(first[-1]) + 1, dtype=torch.float64, device="cuda")
        top = top.scatter_reduce(0, first, part.abs().amax(1), "amax").clamp(min=LEAST)
        over[:, c:c + BLOCK] = part * TOP / top[first][:, None]
        scales.append(top / TOP)
    return {"q": over, "scales": torch.stack(scales, 0 if block_rows == 1 else 1)}


def _exact_act(g, act):
    """act(g) and its slope, in other words than above: silu by tanh, gelu by the logistic function."""
    if act == "silu":
        t = torch.tanh(g / 2)
        return g * (t + 1) / 2, (t + 1) / 2 + g * (1 - t * t) / 4
    a = math.sqrt(8.0 / math.pi)
    p = torch.sigmoid(a * g * (1 + 0.044715 * g * g))
    return g * p, p + g * p * (1 - p) * a * (1 + 0.134145 * g * g)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("rms_norm", "rms_norm_fp8"):
        h = s["x"].double()
        if s["residual"]:
            h = (h + s["other"].double()).to(s["x"].dtype).double()
        rstd = (torch.linalg.vector_norm(h, dim=1) ** 2 / s["n"] + EPS) ** -0.5
        y = s["gamma"].double() * (h * rstd[:, None])
        out = {"rstd": rstd, "sum": h if s["residual"] else None}
        return out | ({"y": y} if op == "rms_norm" else _exact_scaled(y, 1))
    if op == "rms_norm_backward":
        # the Jacobian of h * rstd applied to dy * gamma: one projection taken off
        dy, rstd, h = s["dy"].double(), s["rstd"].double()[:, None], s["x"].double()
        v = dy * s["gamma"].double() * rstd
        dx = v - h * ((v * h).sum(1, keepdim=True) * rstd * rstd / s["n"])
        if s["residual"]:
            dx += s["other"].double()
        return {"dx": dx, "dgamma": torch.mv((h * dy).t(), rstd[:, 0])}
    if op == "quantize_fp8":
        return _exact_scaled(s["x"].double(), s["block_rows"])
    if op == "matmul_fp8":
        y = torch.zeros(s["m"], s["n"], dtype=torch.float64, device="cuda")
        column = torch.arange(s["n"], device="cuda") // BLOCK
        for b, c in enumerate(range(0, s["k"], BLOCK)):
            part = s["x"][:, c:c + BLOCK].double() @ s["w"][:, c:c + BLOCK].double().t().contiguous()
            y += part * s["xs"][b].double()[:, None] * s["ws"][:, b].double()[column]
        return y
    f = s["f"]
    if op == "gated_ffn":
        x, w = s["x"].double(), s["w"].double()
        g, u = x @ w[:, :f], x @ w[:, f:]
        return {"h": u * _exact_act(g, s["act"])[0], "gate_up": torch.cat([g, u], 1) if s["save"] else None}
    g, u = s["gate_up"].double().split(f, 1)
    a, slope = _exact_act(g, s["act"])
    if op == "gated_act":
        return a * u
    if op == "gated_act_fp8":
        return _exact_scaled(a * u, 1)
    dh = s["dh"].double()
    dg, du = slope * u * dh, a * dh
    if op == "gated_act_backward":
        return torch.cat([dg, du], 1)
    w, x = s["w"].double(), s["x"].double()
    return {"dx": dg @ w[:, :f].t() + du @ w[:, f:].t(), "dw": torch.cat([x.t() @ dg, x.t() @ du], 1)}
