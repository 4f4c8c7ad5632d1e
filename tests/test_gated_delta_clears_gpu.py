"""A token whose decay is 0 clears the state, whatever the state holds, against the fp64 oracle.

The oracle takes a cleared state for zeros.  Where its answer is not finite (the tokens before a clear of a state that
is not) the calls' must not be either; elsewhere the bounds of ``test_gated_delta_gpu``."""

import numpy as np
import pytest
import torch

from compressive_memory_transformer_sm_b200 import api
from oracle import gated_delta as G
from tests.test_gated_delta_gpu import BF, DEV, FP, HALF, TOL, forward, make, np64

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def same(got, want):
    a, fin = np64(got), np.isfinite(want)
    assert np.array_equal(np.isfinite(a), fin), f"{(np.isfinite(a) != fin).sum()} of {a.size} finite on one side only"
    a, w = np.where(fin, a, 0), np.where(fin, want, 0)
    assert np.all(np.abs(a - w) <= TOL * np.abs(w).max() + HALF[got.dtype] * np.abs(w) * 1.01)


def check(q, k, v, g, beta, S0):
    with np.errstate(invalid="ignore"):
        wo, wS = G.forward(*map(np64, (q, k, v, g, beta, S0)), q.shape[-1] ** -0.5)
    out, S = forward(q, k, v, g, beta, S0)
    same(out, wo)
    same(S, wS)


def spoil(S0):
    """Heads whose states are all NaN, infinite in some columns, NaN in one element, and finite."""
    S0[:, 0::4] = NAN
    S0[:, 1::4, :, ::3] = INF
    S0[:, 1::4, :, 1::3] = -INF
    S0[:, 2::4, 0, 0] = NAN


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H,L,dk,dv", [(4, 6, 33, 50), (4, 64, 128, 128), (4, 200, 64, 40), (5, 150, 128, 16), (10, 130, 128, 128),
                                       (20, 70, 16, 128)])
def test_forward_clears_a_state_that_is_not_finite(H, L, dk, dv, t):
    """Every kind of state with every place of a clear, and without one (places past the end)."""
    x = make(8, H, H, L, dk, dv, t, seed=21)
    spoil(x[5])
    for b, at in enumerate((0, 3, 15, 16, 37, 63, 64, 100)):
        if at < L:
            for h in range(H):
                x[3][b, h, at] = (-INF, -1e30, -800.0)[h % 3]
                if h % 2 and at + 9 < L:
                    x[3][b, h, at + 9] = -INF
    check(*x)


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("at", [0, 20, 63, 64, 700, 1300])
def test_clears_between_and_inside_segments(at, t):
    """Long enough for segments that run side by side: what each makes of the state before it is joined by products."""
    x = make(1, 2, 2, 2500, 128, 32, t, seed=22)
    x[5][0, 0] = NAN
    x[5][0, 1, :, ::2] = -INF
    x[3][0, 0, at] = -INF
    x[3][0, 1, at + 1] = -1e30
    check(*x)


@pytest.mark.parametrize("L", [8, 200])
def test_a_state_that_no_token_clears_is_kept(L):
    """Decays below what fp32 holds in sum, but of no single token."""
    x = make(1, 4, 4, L, 64, 64, FP, seed=23)
    spoil(x[5])
    x[3][:] = -40.0
    check(*x)


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
def test_step_clears_a_state_that_is_not_finite(t):
    B, H, dk, dv = 6, 4, 128, 50
    q, k, v, g, beta, S0 = make(B, H, 2, 1, dk, dv, t, seed=24)
    spoil(S0)
    g[0], g[1], g[2], g[4, 1:] = -INF, -1e30, -800.0, -INF
    with np.errstate(invalid="ignore"):
        wo, wS = G.forward(*map(np64, (q, k, v, g, beta, S0)), dk ** -0.5)
    S, out = S0.clone(), torch.empty(B, H, dv, dtype=t, device=DEV)
    api.infini_attn_gated_delta_step(*[y[:, :, 0] for y in (q, k, v, g, beta)], S, out)
    same(out, wo[:, :, 0])
    same(S, wS)
