"""The 64-bit definitions of the router and of MXFP4 against hand-worked values,
differences and each other."""
import numpy as np
import pytest

from oracle import ops


def test_top_k_order_ties_and_nan():
    l = np.array([[1.0, 3.0, 3.0, -0.0, 0.0, np.nan, -np.inf, 2.0]])
    assert ops.top_k(l, 8).tolist() == [[1, 2, 7, 0, 3, 4, 6, 5]]


def test_router_by_hand():
    # two tokens, two segments of one token; e^l are 1, 2, 3 and 4, 2, 2
    l = np.log(np.array([[1.0, 2.0, 3.0], [4.0, 2.0, 2.0]]))
    ids, gates, counts, sums, tokens, loss = ops.router(l, 2, 1, "softmax", True, 2.0)
    assert ids.tolist() == [[2, 1], [0, 1]]
    assert np.allclose(gates, [[1.2, 0.8], [4 / 3, 2 / 3]])
    assert counts.tolist() == [[0, 1, 1], [1, 1, 0]] and tokens.tolist() == [1, 1]
    assert np.allclose(sums, [[1 / 6, 1 / 3, 1 / 2], [1 / 2, 1 / 4, 1 / 4]])
    # 3/2 (1/3 + 1/2) and 3/2 (1/2 + 1/4), averaged
    assert np.isclose(loss, (1.25 + 1.125) / 2)


def test_even_routing_has_loss_one():
    l = np.zeros((6, 3))
    q = np.full((6, 3), 1 / 3)
    ids = np.array([[i % 3, (i + 1) % 3] for i in range(6)])
    assert np.isclose(ops.balance(q, ids, np.ones(6, bool), 6)[3], 1.0)
    assert ops.router(l, 2, 6, "sigmoid", True, 1.0, np.zeros(6, bool))[5] == 0.0


def test_all_masked_by_minus_infinity():
    l = np.full((1, 4), -np.inf)
    for kind in ("softmax", "sigmoid"):
        ids, gates, counts, sums, _, loss = ops.router(l, 2, 1, kind, True, 1.0)
        assert ids.tolist() == [[0, 1]] and not gates.any() and not sums.any() and loss == 0


def test_shares_of_vanishing_sigmoids():
    # sigmoid(-2000) is 0 in 64 bits; the shares are those of e^-2000 and e^-2001
    l = np.array([[-2000.0, -2001.0, -3000.0]])
    _, gates, _, sums, _, _ = ops.router(l, 2, 1, "sigmoid", True, 1.0)
    want = np.array([1.0, np.exp(-1.0)]) / (1 + np.exp(-1.0))
    assert np.allclose(gates[0], want) and np.allclose(sums[0, :2], want)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise", [True, False])
def test_gradient_against_differences(kind, normalise):
    rng = np.random.default_rng(1)
    T, E, K, seg, scale, d_loss = 5, 7, 3, 2, 1.7, 2.3
    l = rng.standard_normal((T, E)) * 2
    live = np.array([1, 1, 0, 1, 1], bool)
    dg = rng.standard_normal((T, K))
    ids = ops.top_k(l, K)

    def value(x):
        s, q = ops.scores(x, kind)
        loss = ops.balance(q, ids, live, seg)[3]
        return (dg * ops.gates_of(x, kind, ids, normalise, scale, live)).sum() + d_loss * loss

    grad, size = ops.router_backward(l, ids, seg, kind, normalise, scale, live, dg, d_loss)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            assert abs((value(up) - value(down)) / (2 * h) - grad[t, e]) < 1e-8
    assert (np.abs(grad) <= size * (1 + 1e-9)).all()


def test_gradient_of_rows_with_nan():
    # a sigmoid gate depends on its own logit (normalised: on the chosen ones), the loss and
    # every softmax on the whole row
    l = np.array([[1.0, np.nan, 2.0, 0.5], [np.nan, 1.0, np.nan, np.nan]])
    ids = ops.top_k(l, 2)
    assert ids.tolist() == [[2, 0], [1, 0]]
    dg = np.array([[1.0, 3.0], [1.0, 3.0]])
    slope = lambda x: np.exp(-x) / (1 + np.exp(-x)) ** 2  # noqa: E731
    grad, _ = ops.router_backward(l, ids, 2, "sigmoid", False, 2.0, None, dg, 0.0)
    assert np.allclose(grad[0], [6 * slope(1.0), 0, 2 * slope(2.0), 0])
    assert np.allclose(grad[1], [np.nan, 2 * slope(1.0), 0, 0], equal_nan=True)
    grad, _ = ops.router_backward(l, ids, 2, "sigmoid", True, 2.0, None, dg, 0.0)
    assert np.isfinite(grad[0]).all() and grad[0][[1, 3]].tolist() == [0, 0] and grad[0][0] > 0
    assert np.isnan(grad[1][:2]).all() and grad[1][2:].tolist() == [0, 0]
    for kind, d_loss in (("sigmoid", 1.0), ("softmax", 0.0), ("softmax", 1.0)):
        assert np.isnan(ops.router_backward(l, ids, 2, kind, True, 2.0, None, dg, d_loss)[0]).all()


def test_mxfp4_by_hand():
    x = np.zeros((1, 32))
    # largest 7 = 1.75 2^2: scale 1; ties go to the even code, 7 is cut to 6
    x[0, :12] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.3, -6.9, -0.0, 0.26]
    codes, scales = ops.mxfp4_quantize(x)
    assert scales.tolist() == [[127] + [0] * 15]
    c = np.stack([codes & 15, codes >> 4], -1).reshape(-1)
    assert c[:12].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8 + 1, 8 + 7, 8, 1]
    assert ops.mxfp4_values(codes, scales)[0, :8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]


def test_mxfp4_scales():
    x = np.zeros((1, 160))
    x[0, 0] = 2.0 ** -140          # below every scale: the smallest one, value 0
    x[0, 32] = 6 * 2.0 ** -127     # exponent -125: scale 2^-127
    x[0, 64] = 3 * 2.0 ** 126      # the largest bf16 exponent: scale 2^125
    x[0, 96:98] = [np.nan, 1.0]
    codes, scales = ops.mxfp4_quantize(x)
    assert scales[0, :5].tolist() == [0, 0, 252, 255, 0]
    v = ops.mxfp4_values(codes, scales)
    assert v[0, 0] == 0 and v[0, 32] == 6 * 2.0 ** -127 and v[0, 64] == 3 * 2.0 ** 126
    assert np.isnan(v[0, 96:128]).all() and not v[0, 128:].any()


def test_mxfp4_is_idempotent_and_close():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((8, 96)) * np.exp(rng.standard_normal((8, 1)) * 3)
    v = ops.mxfp4_values(*ops.mxfp4_quantize(x))
    assert np.array_equal(ops.mxfp4_values(*ops.mxfp4_quantize(v)), v)
    top = np.abs(x.reshape(8, 3, 32)).max(-1).repeat(32, -1)
    # half a step of 2 scales, or what is cut above 6 scales: at most a quarter of the largest
    assert (np.abs(v - x) <= top / 4 + 1e-12).all()
