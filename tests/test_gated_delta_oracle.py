"""The fp64 oracle of the gated delta rule and of the layer norm against central finite differences.

With a step of 1e-5 the truncation error is of order 1e-10 and the cancellation error eps / 1e-5 = 2e-11, both
relative to values of order 1 to 10: 1e-7 holds with room."""

import numpy as np
import pytest

from oracle import gated_delta as G

STEP, TOL = 1e-5, 1e-7


def _close(f, x, grad, rng, n=6):
    for _ in range(n):
        at = tuple(int(rng.integers(0, s)) for s in x.shape)
        keep = x[at]
        x[at] = keep + STEP
        up = f()
        x[at] = keep - STEP
        down = f()
        x[at] = keep
        assert abs((up - down) / (2 * STEP) - grad[at]) <= TOL * max(1.0, abs(grad[at]))


@pytest.mark.parametrize("Hk,H,lens", [(2, 2, None), (1, 3, [5, 0]), (2, 4, [3, 7])])
def test_gated_delta_gradients(Hk, H, lens):
    rng = np.random.default_rng(5)
    B, L, dk, dv, scale = 2, 7, 4, 3, 0.7
    q, k = rng.normal(size=(B, Hk, L, dk)), rng.normal(size=(B, Hk, L, dk)) / 2
    v, d_out = rng.normal(size=(2, B, H, L, dv))
    g, beta = -rng.random((B, H, L)), rng.random((B, H, L))
    S0, dS = rng.normal(size=(2, B, H, dk, dv))

    def loss():
        out, S = G.forward(q, k, v, g, beta, S0, scale, lens)
        return float(np.nansum(out * d_out) + np.sum(S * dS))

    grads = G.backward(q, k, v, g, beta, S0, d_out, dS, scale, lens)
    for x, grad in zip((q, k, v, g, beta, S0), grads):
        _close(loss, x, grad, rng)


def test_one_token_by_hand():
    # S' = e^0 * 2 = 2, u = 0.5 * (3 - 2 * 1) = 0.5, S = 2.5, o = 2 * 2.5 * 4
    one = lambda x: np.full((1, 1, 1, 1), float(x))  # noqa: E731
    s = lambda x: np.full((1, 1, 1), float(x))  # noqa: E731
    out, S = G.forward(one(4), one(1), one(3), s(0), s(0.5), one(2), 2.0)
    assert out.item() == 20.0 and S.item() == 2.5
    # a decay of 0 forgets the state before the token
    out, S = G.forward(one(4), one(1), one(3), s(-np.inf), s(0.5), one(2), 2.0)
    assert out.item() == 12.0 and S.item() == 1.5


def test_layer_norm_gradients():
    rng = np.random.default_rng(6)
    x, dy = rng.normal(size=(2, 3, 5))
    w, b = rng.normal(size=(2, 5))
    dx, dw, db = G.layer_norm_backward(x, w, dy, 1e-3)
    loss = lambda: float(np.sum(G.layer_norm(x, w, b, 1e-3) * dy))  # noqa: E731
    for t, grad in ((x, dx), (w, dw), (b, db)):
        _close(loss, t, grad, rng)
