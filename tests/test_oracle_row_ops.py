"""Pins the fp64 definitions of the row operators (oracle/row_ops.py): closed
forms, hand-worked routings, and every gradient against central differences of
the forward it belongs to."""
import numpy as np
import pytest

from oracle import row_ops as R


def differences(f, x, dout, h=1e-6):
    """d<f(x), dout>/dx by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = ((f(up) - f(down)) * dout).sum() / (2 * h)
    return g


def test_layer_norm_of_hand_worked_rows():
    y, mean, rstd = R.layer_norm(np.array([[1.0, 3.0], [5.0, 5.0]]), np.array([2.0, 1.0]), np.array([0.5, 0.0]), 0.0 + 1e-12)
    assert np.allclose(mean, [2.0, 5.0])
    assert np.allclose(y[0], [-2.0 + 0.5, 1.0])
    assert np.allclose(y[1], [0.5, 0.0])
    assert np.isclose(rstd[1], 1e6)


def test_layer_norm_gradient_is_the_differences():
    g = np.random.default_rng(1)
    x, gamma, beta, dy, ds = (g.standard_normal(s) for s in ((4, 7), 7, 7, (4, 7), (4, 7)))
    fwd = lambda x_, ga, be: R.layer_norm(x_, ga, be, 1e-3)[0]  # noqa: E731
    _, mean, rstd = R.layer_norm(x, gamma, beta, 1e-3)
    dx, dg, db = R.layer_norm_backward(dy, x, gamma, mean, rstd, ds)
    assert np.allclose(dx, differences(lambda v: fwd(v, gamma, beta), x, dy) + ds, atol=1e-7)
    assert np.allclose(dg, differences(lambda v: fwd(x, v, beta), gamma, dy), atol=1e-7)
    assert np.allclose(db, differences(lambda v: fwd(x, gamma, v), beta, dy), atol=1e-7)


def test_embedding_and_its_gradient():
    g = np.random.default_rng(2)
    ids = np.array([3, 9, 4, 3, -1, 7, 3])
    table, dy = g.standard_normal((4, 3)), g.standard_normal((7, 3))
    y = R.embedding(ids, table, 3, 2.0)
    onehot = (ids[:, None] - 3 == np.arange(4)).astype(float)
    assert np.array_equal(y, 2.0 * (onehot @ table))
    assert np.allclose(R.embedding_grad(ids, dy, 4, 3, 2.0), 2.0 * (onehot.T @ dy))
    assert np.allclose(R.embedding_grad(ids, dy, 4, 3, 2.0), differences(lambda v: R.embedding(ids, v, 3, 2.0), table, dy),
                       atol=1e-7)


def test_router_of_a_hand_worked_batch():
    # 4 tokens, 4 experts, 2 destinations of 2, 2 pieces; token 2 is padding
    x = np.log(np.array([[0.1, 0.6, 0.1, 0.2], [0.4, 0.1, 0.4, 0.1], [0.25] * 4, [0.7, 0.1, 0.1, 0.1]]))
    r = R.moe_router(x, 2, 2, 2, 0.5, False, mask=[1, 1, 0, 1])
    assert r["ids"].tolist() == [[1, 3], [0, 2], [-1, -1], [0, 1]]
    assert r["counts"].tolist() == [[1, 1, 1, 1], [1, 1, 0, 0]]
    # destination 0: piece 0 experts 0, 1, then piece 1; destination 1: piece 0
    assert r["positions"].tolist() == [[1, 5], [0, 4], [-1, -1], [2, 3]]
    assert np.allclose(r["gates"], [[0.6, 0.2], [0.4, 0.4], [0, 0], [0.7, 0.1]])
    assert r["valid"] == 3 and np.allclose(r["prob_sums"], [1.2, 0.8, 0.6, 0.4])
    assert np.isclose(r["loss"], 0.5 * 4 / (2 * 9) * (2 * 1.2 + 2 * 0.8 + 0.6 + 0.4))
    assert np.allclose(R.moe_router(x, 2, 2, 2, 0.5, True, mask=[1, 1, 0, 1])["gates"][0], [0.75, 0.25])


def test_router_empty_rows_and_order():
    inf = np.inf
    x = np.array([[-inf, -inf, -inf], [-inf, 2.0, -inf], [1.0, np.nan, inf], [0.0, 0.0, 0.0]])
    r = R.moe_router(x, 2, 1, 1, 1.0, True)
    assert r["ids"].tolist() == [[-1, -1], [1, -1], [1, 2], [0, 1]]
    assert r["valid"] == 3 and np.isnan(r["loss"])
    assert R.moe_router(x[:1], 2, 1, 1, 1.0, True)["loss"] == 0.0


def test_balanced_routing_has_loss_coef():
    """Uniform probabilities and equal counts: the loss is its least value, coef."""
    experts = 4
    x = np.zeros((experts, experts)) + 1e-9 * np.eye(experts)
    assert np.isclose(R.moe_router(x, 1, 1, 1, 0.3, False)["loss"], 0.3)


@pytest.mark.parametrize("renormalize", [False, True])
def test_router_gradient_is_the_differences(renormalize):
    g = np.random.default_rng(3)
    x = g.standard_normal((5, 6))
    x[2, 4] = -np.inf
    mask = [1, 1, 1, 0, 1]
    dg, dl, coef = g.standard_normal((5, 3)), 1.7, 0.4
    r = R.moe_router(x, 3, 2, 2, coef, renormalize, mask)

    def value(v):
        s = R.moe_router(v, 3, 2, 2, coef, renormalize, mask)
        assert np.array_equal(s["ids"], r["ids"])    # the steps change no choice
        return np.array((s["gates"] * dg).sum() + dl * s["loss"])

    got = R.moe_router_backward(x, r["ids"], r["counts"], dg, dl, coef, renormalize, mask)
    finite = np.isfinite(x)
    with np.errstate(invalid="ignore"):
        want = differences(value, x, 1.0)
    assert np.allclose(got[finite], want[finite], atol=1e-7)
    assert not got[~finite].any() and not got[3].any()


def test_combine_and_its_gradient():
    g = np.random.default_rng(4)
    h, gates, dy = g.standard_normal((5, 3)), g.standard_normal((3, 2)), g.standard_normal((3, 3))
    pos = np.array([[4, 0], [-1, 2], [-1, 9]])
    y = R.moe_combine(h, pos, gates)
    assert np.allclose(y, [gates[0, 0] * h[4] + gates[0, 1] * h[0], gates[1, 1] * h[2], np.zeros(3)])
    dh, dgates = R.moe_combine_backward(dy, h, pos, gates)
    assert np.allclose(dh, differences(lambda v: R.moe_combine(v, pos, gates), h, dy), atol=1e-7)
    assert np.allclose(dgates, differences(lambda v: R.moe_combine(h, pos, v), gates, dy), atol=1e-7)
    assert np.array_equal(R.moe_combine(h, pos), R.moe_combine(h, pos, np.ones((3, 2))))
