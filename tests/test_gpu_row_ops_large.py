"""The row operators at offsets past 2^32 bytes: the rows' own results in a
small call, bit for bit."""
import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests._util import log
from tests.test_gpu_row_ops import equal

pytestmark = pytest.mark.gpu

ROWS, N = 131071, 16383   # just below 2^31 elements, of 4 bytes
NAMED = [ROWS - 1, 70000, 65536, 3]


def dense(*shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(len(shape)), device="cuda")


def test_combine_backward_of_a_large_matrix_of_rows():
    """h and dh."""
    h, dh = torch.empty(ROWS, N, device="cuda"), torch.zeros(ROWS, N, device="cuda")
    small = dense(len(NAMED), N)
    h[NAMED] = small
    dy, gates = dense(2, N), torch.rand(2, 2, device="cuda")
    pos = torch.tensor(NAMED, dtype=torch.int32, device="cuda").view(2, 2)
    _, dg = tgc.moe_combine_backward(dy, h, pos, gates, dh=dh)
    want, want_dg = tgc.moe_combine_backward(dy, small, torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2),
                                             gates)
    equal(dh[NAMED], want, "dh")
    equal(dg, want_dg, "dgates")
    assert not dh[4:65536].any() and not dh[70001:ROWS - 1].any()


def test_row_moves_of_many_tokens():
    """The tokens' side: x of permute, y of combine, dy of its gradient."""
    x = torch.empty(ROWS, N, device="cuda")
    small = dense(len(NAMED), N)
    x[NAMED] = small
    pos = torch.full((ROWS, 1), -1, dtype=torch.int32, device="cuda")
    pos[NAMED, 0] = torch.arange(4, dtype=torch.int32, device="cuda")
    rows = tgc.moe_permute(x, pos, 4)
    equal(rows, small, "permute")
    gates = torch.rand(ROWS, 1, device="cuda")
    own = torch.arange(4, dtype=torch.int32, device="cuda").view(4, 1)
    dh, dg = tgc.moe_combine_backward(x, rows, pos, gates)
    want, want_dg = tgc.moe_combine_backward(small, rows, own, gates[NAMED])
    equal(dh, want, "dh")
    equal(dg[NAMED], want_dg, "dgates")
    y = tgc.moe_combine(rows, pos, gates, y=x)
    equal(y[NAMED], tgc.moe_combine(rows, own, gates[NAMED]), "combine")
    assert not y[70001:ROWS - 1].any()


def test_embedding_of_many_tokens():
    """y of the lookup, dy of its gradient."""
    ids = torch.full((ROWS,), 50, device="cuda")
    ids[NAMED] = torch.tensor([2, 0, 2, 1], device="cuda")
    table = dense(3, N)
    y = tgc.embedding(ids, table, scale=3.0)
    equal(y[NAMED], tgc.embedding(ids[NAMED], table, scale=3.0), "lookup")
    assert not y[70001:ROWS - 1].any()
    # the order of a row's tokens is theirs in the batch
    order = sorted(NAMED)
    equal(tgc.embedding_grad(ids, y, 3), tgc.embedding_grad(ids[order], y[order], 3), "gradient")


def test_layer_norm_of_many_rows():
    rows, n = 65535, 32767
    x = torch.empty(rows, n, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    ga = torch.rand(n, device="cuda")
    y, mean, rstd = tgc.layer_norm(x, ga)
    last = x[-3:].contiguous()
    want = tgc.layer_norm(last, ga)
    for a, b, f in zip((y, mean, rstd), want, ("y", "mean", "rstd")):
        equal(a[-3:].contiguous(), b, f)
    dx = tgc.layer_norm_backward(x, x, ga, mean, rstd, dx=y)[0]
    equal(dx[-3:].contiguous(), tgc.layer_norm_backward(last, last, ga, want[1], want[2])[0], "dx")


@pytest.mark.parametrize("tokens,ld", [(65, 33000000), (70000, 30000)])   # one workgroup; many
def test_router_of_widely_strided_logits(tokens, ld):
    log(f"router of {tokens} rows {ld} apart")
    experts, topk = 96, 4
    small = dense(tokens, experts)
    store = torch.empty((tokens - 1) * ld + experts, device="cuda")
    x = store.as_strided((tokens, experts), (ld, 1))
    x.copy_(small)
    got, want = tgc.moe_router(x, topk, pieces=2, world=2), tgc.moe_router(small, topk, pieces=2, world=2)
    for a, b, f in zip(got, want, got._fields):
        equal(a, b, f)
    dg, dl = dense(tokens, topk), torch.ones(1, device="cuda")
    out = torch.empty_like(store).as_strided((tokens, experts), (ld, 1))
    tgc.moe_router_backward(x, got.ids, got.gates, got.counts, got.valid, dg, dl, dlogits=out)
    equal(out.contiguous(), tgc.moe_router_backward(small, got.ids, got.gates, got.counts, got.valid, dg, dl), "dlogits")
