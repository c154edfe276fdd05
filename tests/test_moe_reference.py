"""The 64-bit statements of the mixture-of-experts operators against closed
forms, the oracle and central differences; no GPU."""
import numpy as np
import pytest

import moe_reference as ref
import oracle
import synth


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_grad_matches_differences(score, renormalize):
    rng = np.random.default_rng(5)
    x, g = rng.normal(size=(6, 11)), rng.normal(size=(6, 4))
    x[2, 3] = -np.inf
    _, ids = ref.route(x, 4, score)
    ids[4, 3] = -1
    got = ref.route_grad(x, ids, g, score, renormalize, 1.7)
    h = 1e-6
    for e in range(11):
        up, down = x.copy(), x.copy()
        up[:, e] += h
        down[:, e] -= h
        d = (ref.route_weights(up, ids, score, renormalize, 1.7) - ref.route_weights(down, ids, score, renormalize, 1.7)) / (2 * h)
        # central difference: h^2 / 6 times a third derivative of order one, and 1e-16 / h of rounding
        np.testing.assert_allclose(got[:, e], (d * np.where(ids >= 0, g, 0.0)).sum(1), atol=2e-9)


def test_combine_grad_matches_differences():
    rng = np.random.default_rng(6)
    h, w, gy = rng.normal(size=(3, 4, 5)), rng.normal(size=(3, 4)), rng.normal(size=(3, 5))
    ids = np.array([[0, 1, -1, 2], [3, 2, 1, 0], [-1, -1, -1, -1]])
    gh, gw = ref.combine_grad(gy, h, w, ids)
    loss = lambda hh, ww: (ref.combine(hh, ww, ids) * gy).sum()
    for t in range(3):
        for j in range(4):
            d = np.zeros_like(w)
            d[t, j] = 0.5
            assert abs(loss(h, w + d) - loss(h, w - d) - gw[t, j]) < 1e-12      # linear in w and in h
            d = np.zeros_like(h)
            d[t, j, 2] = 0.5
            assert abs(loss(h + d, w) - loss(h - d, w) - gh[t, j, 2]) < 1e-12


def test_mxfp4_round_is_the_quantize_rule():
    w, bits = synth.normal((9, 256), 1.0, 91, synth.WEIGHT, "f32")
    wq, sc, _ = oracle.quantize(bits, "f32", 32, 4, "mxfp4")
    np.testing.assert_array_equal(ref.mxfp4_round(w.double().numpy()), ref.mxfp4_decode(wq, sc))


def test_route_ties_and_closed_form():
    x = np.array([[1.0, 2.0, 2.0, -np.inf, np.nan, 2.0]])
    w, ids = ref.route(x, 5)
    assert ids.tolist() == [[1, 2, 5, 0, -1]]
    e = np.exp(-1.0)
    np.testing.assert_allclose(w[0], np.array([1, 1, 1, e, 0]) / (3 + e), rtol=1e-15)
