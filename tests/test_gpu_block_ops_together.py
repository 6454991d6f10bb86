"""The gated feed-forward block's operators called at once from several threads and
streams, in two graphs that are replayed at once, and on tensors at addresses that are
aligned to their elements alone: every result has the bits of a call by itself."""
import threading

import pytest
import torch

import tensor_gemm_collective_amd as tgc
from tests.test_gpu_block_ops import block_state, whole_pass
from tests.test_gpu_row_ops import equal

pytestmark = pytest.mark.gpu


def same(got, want, what):
    for k, (a, b) in enumerate(zip(got, want)):
        equal(a, b, f"{what}, output {k}")


def test_threads_with_their_own_streams():
    states = [block_state(i) for i in range(3)]
    want = [whole_pass(s) for s in states]
    torch.cuda.synchronize()
    got, errors = [None] * 3, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    got[i] = whole_pass(states[i])
            stream.synchronize()
        except Exception as e:   # shown below, by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(3):
        same(got[i], want[i], f"thread {i}")


def test_errors_belong_to_their_thread():
    x = torch.ones(2, 24, device="cuda")
    seen = []

    def work():
        with pytest.raises(tgc.CocError):
            tgc.quantize_fp8(x)
        seen.append(tgc.lib().coc_last_error())

    t = threading.Thread(target=work)
    t.start()
    t.join()
    tgc.rms_norm(x, x[0].contiguous())
    assert b"multiple of 16" in seen[0] and tgc.lib().coc_last_error() == b""


def test_two_graphs_replayed_at_once():
    states = [block_state(i) for i in range(2)]
    want = [whole_pass(s) for s in states]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in states:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            whole_pass(s)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(whole_pass(s))
        graphs.append(g)
    torch.cuda.synchronize()
    for turn in range(4):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            same(outs[i], want[i], f"replay {turn} of graph {i}")
        whole_pass(states[0])


def moved(t, by):
    """t's values in memory that begins `by` elements into an allocation."""
    big = torch.empty(t.numel() + by + 8, dtype=t.dtype, device=t.device)
    to = big[by:by + t.numel()].view(t.shape)
    to.copy_(t)
    return to


@pytest.mark.parametrize("by", [1, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_addresses_aligned_to_elements(dtype, by):
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, dh, gamma, res = n(130, 544), n(130, 272), n(544), n(130, 544)
    odd = [moved(t, by) for t in (x, dh, gamma, res)]
    assert odd[0].data_ptr() % 16
    for rows in (1, 128):
        same(tgc.quantize_fp8(odd[0], block_rows=rows), tgc.quantize_fp8(x, block_rows=rows), "quantize")
    same(tgc.gated_act_fp8(odd[0]), tgc.gated_act_fp8(x), "activation in 8 bits")
    same(tgc.rms_norm_fp8(odd[0], odd[2], residual=odd[3]), tgc.rms_norm_fp8(x, gamma, residual=res), "norm in 8 bits")
    h, d = moved(dh, by), moved(x, by)
    tgc.gated_act(odd[0], act="gelu", h=h)
    tgc.gated_act_backward(odd[1], odd[0], act="gelu", dgate_up=d)
    equal(h, tgc.gated_act(x, act="gelu"), "activation")
    equal(d, tgc.gated_act_backward(dh, x, act="gelu"), "its gradient")
    q, qs = tgc.quantize_fp8(x)
    w, ws = tgc.quantize_fp8(n(256, 544), block_rows=128)
    for m in (1, 20, 130):
        s = qs[:, :m].contiguous()
        y = moved(n(m, 256), by)
        tgc.matmul_fp8(q[:m], s, w, ws, y=y)
        equal(y, tgc.matmul_fp8(q[:m], s, w, ws, dtype=dtype), f"product of {m} rows")
