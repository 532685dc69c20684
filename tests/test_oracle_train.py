"""The float64 definitions of the training and adapter operators: gradients
against central differences, and the losses' fixed points (CPU)."""
import numpy as np
import pytest

from oracle import train as OT

H = 1e-5


def _routing(rng, T, E, k):
    logits = rng.standard_normal((T, E))
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    return logits, ids


def _weights(logits, ids):
    return OT.softmax(np.take_along_axis(logits, ids, axis=1))[0]


@pytest.mark.parametrize("offsets,masked", [(None, False), ([0, 3, 3, 9], True), ([2, 5, 8], False)])
def test_router_gradient_is_the_losses_difference(offsets, masked):
    rng = np.random.default_rng(5)
    T, E, k = 9, 7, 3
    logits, ids = _routing(rng, T, E, k)
    mask = (rng.random(T) > 0.3).astype(np.uint8) if masked else None
    dl, dw = rng.standard_normal(2), rng.standard_normal((T, k))
    r = OT.router_loss(logits, ids, offsets, mask)
    spans, inside = OT.sequences(T, offsets, mask)
    live = np.concatenate([t for _, t in spans])

    def goal(z):
        # the counts stay as they are: only the probabilities move
        q = OT.router_loss(z, ids, offsets, mask)["losses"]
        return dl @ q + (dw * _weights(z, ids))[live].sum()

    g, mag = OT.router_backward(logits, ids, offsets, mask, _weights(logits, ids), dw, dl, r["counts"],
                                r["seq_tokens"])
    for t in range(T):
        if not inside[t]:
            assert np.isnan(g[t]).all()
            continue
        for e in range(E):
            d = np.zeros_like(logits)
            d[t, e] = H
            # central differences: H^2 times a third derivative of order 10, and 2^-52 / H of the goal's size
            assert abs((goal(logits + d) - goal(logits - d)) / (2 * H) - g[t, e]) < 1e-8
    assert (np.abs(np.nan_to_num(g)) <= mag + 1e-15).all()


def test_balance_is_one_for_even_use():
    E, k = 6, 2
    ids = np.array([[0, 1], [2, 3], [4, 5]])
    r = OT.router_loss(np.zeros((3, E)), ids)
    assert np.isclose(r["losses"][0], 1.0) and np.isclose(r["losses"][1], np.log(E) ** 2)
    assert (r["counts"] == 1).all() and list(r["seq_tokens"]) == [3, 3, 1]
    # all tokens on one expert that is expected with certainty: E / k of f, probability 1
    z = np.full((4, E), -np.inf)
    z[:, 2] = 0.0
    r = OT.router_loss(z, np.full((4, 1), 2))
    assert np.isclose(r["losses"][0], E) and r["losses"][1] == 0.0


def test_rows_without_logits_have_no_part():
    z = np.array([[0.0, 1.0, 2.0], [-np.inf, np.nan, -np.inf]])
    ids = np.array([[2], [0]])
    r = OT.router_loss(z, ids)
    assert np.isfinite(r["losses"]).all() and r["counts"].tolist() == [[1, 0, 1]]
    g, _ = OT.router_backward(z, ids, weights=np.ones((2, 1)), dweights=np.ones((2, 1)),
                              dlosses=np.ones(2), counts=r["counts"], seq_tokens=r["seq_tokens"])
    assert (g[1] == 0).all() and np.isfinite(g).all()


def test_finalize_gradient_is_a_difference():
    rng = np.random.default_rng(6)
    T, k, C = 4, 3, 5
    w, y2 = rng.standard_normal((T, k)), rng.standard_normal((T * k, C))
    rows = rng.permutation(T * k).reshape(T, k)
    dout = rng.standard_normal((T, C))
    goal = lambda w, y: ((w[:, :, None] * y[rows]).sum(1) * dout).sum()  # noqa: E731
    dw, _, dy = OT.finalize_backward(dout, w, y2, rows)
    for t in range(T):
        for j in range(k):
            d = np.zeros_like(w)
            d[t, j] = H
            assert abs((goal(w + d, y2) - goal(w - d, y2)) / (2 * H) - dw[t, j]) < 1e-8
            d = np.zeros_like(y2)
            d[rows[t, j], 1] = H
            assert abs((goal(w, y2 + d) - goal(w, y2 - d)) / (2 * H) - dy[t, j, 1]) < 1e-8


def test_adapter_gradients_are_differences():
    rng = np.random.default_rng(7)
    T, L, R, K, N = 6, 3, 2, 4, 5
    x, a, b = rng.standard_normal((T, K)), rng.standard_normal((L, R, K)), rng.standard_normal((L, R, N))
    s, ids = rng.standard_normal(L), np.array([0, 2, -1, 2, 0, 7])
    dout, base = rng.standard_normal((T, N)), rng.standard_normal((T, N))
    goal = lambda x, a, b: (OT.adapter_apply(x, ids, a, b, s, base) * dout).sum()  # noqa: E731
    dx, da, db = OT.adapter_backward(dout, x, ids, a, b, s, np.zeros((T, K)))
    for grad, at in ((dx, 0), (da, 1), (db, 2)):
        args = [x, a, b]
        for i in np.ndindex(grad.shape):
            up, down = list(args), list(args)
            d = np.zeros_like(args[at])
            d[i] = H
            up[at], down[at] = args[at] + d, args[at] - d
            assert abs((goal(*up) - goal(*down)) / (2 * H) - grad[i]) < 1e-7
    assert (da[1] == 0).all() and (db[1] == 0).all() and (dx[2] == 0).all()
