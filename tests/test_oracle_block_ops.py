"""Pins of oracle/block_ops.py: library conversions, closed forms, gradients
against differences, identities."""
import numpy as np
import pytest
import torch

from oracle import block_ops as B


def test_e4m3_rounding_is_the_formats():
    """Against torch's conversion: every 8-bit value, the points half way between
    neighbours and their neighbours, and 200k random values."""
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    values = np.unique(codes[np.isfinite(codes)])
    assert values.max() == 448 and values[values > 0].min() == 2.0 ** -9
    assert np.array_equal(B.round_e4m3(values), values)
    mid = (values[1:] + values[:-1]) / 2
    g = np.random.default_rng(0)
    x = np.concatenate([mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)),
                        np.nextafter(mid.astype(np.float32), np.float32(-1e9)),
                        g.uniform(-448, 448, 100000), g.standard_normal(100000) * 2.0 ** g.integers(-12, 7, 100000)])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(B.round_e4m3(x.astype(np.float64)), want)


def test_quantized_blocks():
    """One value a block: it is stored as 448 (its sign kept) and reads back as
    itself; zeros as zeros; each block has its own scale."""
    y = np.zeros((3, 300))
    y[0, 5], y[0, 200], y[2, 299] = 7.0, -2.0 ** -50, 1e30
    q, s = B.quantize(y, 1)
    assert s.shape == (3, 3) and np.array_equal(q != 0, y != 0) and set(np.abs(q[q != 0])) == {448.0}
    assert np.allclose(q * B.spread(s, 1, y.shape), y, rtol=1e-15, atol=0)
    assert s[1, 0] == 2.0 ** -96 / 448
    q, s = B.quantize(y, 128)
    assert s.shape == (1, 3) and np.array_equal(s[0] * 448, [7.0, 2.0 ** -50, 1e30])


def test_matmul_fp8_is_the_product_of_what_it_stands_for():
    g = np.random.default_rng(1)
    y, z = g.standard_normal((5, 272)), g.standard_normal((140, 272))
    (q, s), (p, t) = B.quantize(y, 1), B.quantize(z, 128)
    want = (q * B.spread(s, 1, y.shape)) @ (p * B.spread(t, 128, z.shape)).T
    assert np.allclose(B.matmul_fp8(q, s.T, p, t), want, rtol=1e-12, atol=1e-12)
    # one hot: a row of w times its scale
    one = np.zeros((1, 272))
    one[0, 260] = 1.0
    assert np.array_equal(B.matmul_fp8(one, np.ones((3, 1)), p, t)[0], p[:, 260] * np.repeat(t[:, 2], 128)[:140])


def test_rms_norm_closed_forms():
    y, r = B.rms_norm(np.array([[3.0, -4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(r, 1 / np.sqrt(12.5)) and np.allclose(y, [[3 / np.sqrt(12.5), -8 / np.sqrt(12.5)]])
    y, r = B.rms_norm(np.zeros((1, 4)), np.ones(4), 4.0)
    assert r[0] == 0.5 and not y.any()


def difference(f, x, d, eps=1e-6):
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


def test_rms_norm_gradient_against_differences():
    g = np.random.default_rng(2)
    h, gamma, dy, ds = g.standard_normal((3, 17)), 1 + 0.2 * g.standard_normal(17), *g.standard_normal((2, 3, 17))
    rstd = B.rms_norm(h, gamma, 1e-3)[1]
    dx, dg = B.rms_norm_backward(dy, h, gamma, rstd, ds)
    d = g.standard_normal((3, 17))
    loss = lambda v: (B.rms_norm(v, gamma, 1e-3)[0] * dy).sum() + (v * ds).sum()  # noqa: E731
    assert np.isclose(difference(loss, h, d), (dx * d).sum(), rtol=1e-7)
    e = g.standard_normal(17)
    assert np.isclose(difference(lambda v: (B.rms_norm(h, v, 1e-3)[0] * dy).sum(), gamma, e), (dg * e).sum(), rtol=1e-7)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activations(kind):
    g = np.linspace(-9, 9, 181)
    a, s = B.act(g, kind)
    t = torch.from_numpy(g)
    want = torch.nn.functional.silu(t) if kind == "silu" else torch.nn.functional.gelu(t, approximate="tanh")
    assert np.allclose(a, want.numpy(), rtol=1e-13, atol=1e-15)
    assert np.allclose(s, (B.act(g + 1e-6, kind)[0] - B.act(g - 1e-6, kind)[0]) / 2e-6, atol=1e-9)
    assert B.act(np.zeros(1), kind)[0][0] == 0 and B.act(np.zeros(1), kind)[1][0] == 0.5


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_gradients_against_differences(kind):
    g = np.random.default_rng(3)
    x, w, dh = g.standard_normal((4, 6)), g.standard_normal((6, 10)), g.standard_normal((4, 5))
    h, both = B.gated_ffn(x, w, kind)
    assert np.allclose(h[2, 3], B.act(both[2, 3], kind)[0] * both[2, 8])
    dx, dw = B.gated_ffn_backward(dh, x, w, both, kind)
    loss = lambda a, b: (B.gated_ffn(a, b, kind)[0] * dh).sum()  # noqa: E731
    d, e = g.standard_normal(x.shape), g.standard_normal(w.shape)
    assert np.isclose(difference(lambda v: loss(v, w), x, d), (dx * d).sum(), rtol=1e-7)
    assert np.isclose(difference(lambda v: loss(x, v), w, e), (dw * e).sum(), rtol=1e-7)
