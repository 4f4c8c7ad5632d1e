"""fp64 CPU oracle for the gated delta rule and layer normalisation, and their gradients.

TEST INFRASTRUCTURE ONLY, like ``infini_ref``: nothing on the product path imports it.

The recurrence is taken token by token from its definition ("Gated Delta Networks: Improving
Mamba2 with Delta Rule", arXiv 2412.06464, Eq. 10), the gradients from the chain rule over the
same steps; both are pinned to central finite differences, not to themselves.
"""

from __future__ import annotations

import numpy as np


def forward(q, k, v, g, beta, S0, scale, lens=None):
    """q, k [B,Hk,L,dk], v [B,H,L,dv], g, beta [B,H,L], S0 [B,H,dk,dv]: (out, S); rows past lens[b] of out are NaN."""
    B, H, L = g.shape
    group = H // q.shape[1]
    out = np.full(v.shape, np.nan)
    S = S0.copy()
    for b in range(B):
        for h in range(H):
            M = S[b, h]
            for t in range(L if lens is None else min(max(int(lens[b]), 0), L)):
                kt, qt = k[b, h // group, t], q[b, h // group, t]
                M = np.exp(g[b, h, t]) * M if np.exp(g[b, h, t]) > 0 else np.zeros_like(M)
                M = M + np.outer(kt, beta[b, h, t] * (v[b, h, t] - kt @ M))
                out[b, h, t] = scale * (qt @ M)
            S[b, h] = M
    return out, S


def backward(q, k, v, g, beta, S0, d_out, dS, scale, lens=None):
    """Gradients (dq, dk, dv, dg, dbeta, dS0) of sum(out * d_out) + sum(S_L * dS)."""
    B, H, L = g.shape
    group = H // q.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dg, db, dS0 = np.zeros(g.shape), np.zeros(g.shape), np.zeros(S0.shape)
    for b in range(B):
        n = L if lens is None else min(max(int(lens[b]), 0), L)
        for h in range(H):
            hk = h // group
            M, kept = S0[b, h], []
            for t in range(n):
                kept.append(M)
                D = np.exp(g[b, h, t]) * M
                M = D + np.outer(k[b, hk, t], beta[b, h, t] * (v[b, h, t] - k[b, hk, t] @ D))
            G = dS[b, h].copy()
            for t in reversed(range(n)):
                a, be, kt, qt = np.exp(g[b, h, t]), beta[b, h, t], k[b, hk, t], q[b, hk, t]
                P = kept[t]
                D = a * P
                e = v[b, h, t] - kt @ D
                dq[b, hk, t] += scale * (M @ d_out[b, h, t])
                G = G + scale * np.outer(qt, d_out[b, h, t])
                du = kt @ G
                db[b, h, t] = du @ e
                dv[b, h, t] = be * du
                dk[b, hk, t] += G @ (be * e) - be * (D @ du)
                G = G - np.outer(kt, be * du)
                dg[b, h, t] = a * np.sum(G * P)
                G = a * G
                M = P
            dS0[b, h] = G
    return dq, dk, dv, dg, db, dS0


def layer_norm(x, w, bias, eps):
    d = x - x.mean(-1, keepdims=True)
    y = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps) * w
    return y if bias is None else y + bias


def layer_norm_backward(x, w, dy, eps):
    """(dx, dweight, dbias) of sum(layer_norm(x) * dy)."""
    d = x - x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    z, h = d * rstd, dy * w
    dx = rstd * (h - h.mean(-1, keepdims=True) - z * (h * z).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, (dy * z).sum(axes), dy.sum(axes)
