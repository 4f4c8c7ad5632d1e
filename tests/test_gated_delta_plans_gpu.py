"""The kernels that many heads, few long sequences and long tensors select, against the recurrence in 64 bits.

Every case names the state kernels it is for, and the test asserts that they ran: o (outputs), s (segments of the
forward), B (both passes of the backward) and S (its segments), each with the warps that share 16 value columns.

Bounds.  Elementwise as in ``test_gated_delta_gpu``.  For fp32 results also relative in the L2 norm: a product is at
most 8 steps of 16 terms, each of which may truncate the running sum by 2^-23 of it; truncations are spread evenly, so
that their mean, which is what remains of them in a sum, is 2^-24 each: 8 * 2^-24 = 2^-21 a product if all have one
sign.  A result is at the end of four products (K S, T X, K^T U and its own): 4 * 2^-21 = 2^-19 = 1.9e-6, and what
earlier chunks left decays.  Values of two bf16 parts instead of three are off by up to 2^-8 of a remainder of up to
2^-8, 2^-16 = 1.5e-5, and about 2.6e-6 in the mean square: X or rho U in two parts does not meet the bound."""

import re

import numpy as np
import pytest
import torch

from compressive_memory_transformer_sm_b200 import api
from oracle import gated_delta as G
from tests.test_gated_delta_gpu import BF, DEV, FP, backward_inputs, forward, make, near, np64

L2 = 2.0 ** -19
gpu = pytest.mark.gpu
types = pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])


def reference(x, scale, lens=None, d_out=None, dS=None):
    """(out, S) and, with d_out, the gradients: every (b, h) at once, token by token, in 64 bits on the inputs' device.
    Rows of out past lens[b] are NaN."""
    q, k, v, g, beta, S = (y.double() for y in x)
    B, H, L = g.shape
    group, shape = H // q.shape[1], S.shape
    n = torch.full((B,), L, device=q.device) if lens is None else lens.long().clamp(0, L)
    live = (torch.arange(L, device=q.device)[:, None] < n)[:, :, None].expand(L, B, H).reshape(L, B * H)
    rows = lambda y: torch.where(live[..., None], y.movedim(2, 0).reshape(L, B * H, -1), 0.)  # noqa: E731
    heads = lambda y: rows(y.repeat_interleave(group, 1))  # noqa: E731
    q, k, v = heads(q), heads(k), rows(v)
    a = torch.where(live, torch.exp(g).movedim(2, 0).reshape(L, -1), 1.)[..., None, None]
    be = torch.where(live, beta.movedim(2, 0).reshape(L, -1), 0.)[..., None]
    S, kept, out = S.reshape(B * H, *shape[2:]), [], []
    dot = lambda y, M: torch.bmm(y[:, None], M)[:, 0]  # noqa: E731
    for t in range(L):
        if d_out is not None:
            kept.append(S)
        S = S * a[t]
        S = torch.baddbmm(S, k[t][:, :, None], (be[t] * (v[t] - dot(k[t], S)))[:, None])
        out.append(dot(q[t], S))
    back = lambda y: y.reshape(L, B, H, *y.shape[2:]).movedim(0, 2)  # noqa: E731
    o = back(torch.where(live[..., None], scale * torch.stack(out), float("nan")))
    if d_out is None:
        return o, S.view(shape)
    d, D = scale * rows(d_out.double()), torch.zeros_like(S) if dS is None else dS.double().reshape(S.shape)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(be[..., 0]), torch.zeros_like(be[..., 0])
    end = S
    for t in reversed(range(L)):
        P, after = kept[t], S
        M = P * a[t]
        e = v[t] - dot(k[t], M)
        dq[t] = torch.bmm(after, d[t][:, :, None])[:, :, 0]
        D = torch.baddbmm(D, q[t][:, :, None], d[t][:, None])
        du = dot(k[t], D)
        db[t], dv[t] = (du * e).sum(-1), be[t] * du
        dk[t] = torch.bmm(D, (be[t] * e)[:, :, None])[:, :, 0] - torch.bmm(M, dv[t][:, :, None])[:, :, 0]
        D = torch.baddbmm(D, k[t][:, :, None], -dv[t][:, None])
        dg[t] = a[t, :, 0, 0] * (D * P).sum((1, 2))
        D, S = a[t] * D, P
    shared = lambda y: back(torch.where(live[..., None], y, 0.)).reshape(B, H // group, group, L, -1).sum(2)  # noqa: E731
    mask = lambda y: back(torch.where(live, y, 0.))  # noqa: E731
    return o, end.view(shape), (shared(dq), shared(dk), back(dv), mask(dg), mask(db), D.view(shape))


@pytest.mark.parametrize("lens", [None, [9, 0]])
def test_reference(lens):
    """The reference of this file is the oracle's recurrence."""
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x = (r(2, 2, 13, 5), 0.5 * r(2, 2, 13, 5), r(2, 6, 13, 4), -r(2, 6, 13).abs(), r(2, 6, 13).sigmoid(), r(2, 6, 5, 4))
    d_out, dS = r(2, 6, 13, 4), r(2, 6, 5, 4)
    got = reference(x, 0.3, None if lens is None else torch.tensor(lens), d_out, dS)
    o, S = G.forward(*(y.numpy() for y in x), 0.3, lens)
    want = (o, S, *G.backward(*(y.numpy() for y in x), d_out.numpy(), dS.numpy(), 0.3, lens))
    for a, w in zip((got[0], got[1], *got[2]), want):
        assert a.shape == w.shape and np.allclose(a.numpy(), w, rtol=1e-11, atol=1e-11, equal_nan=True)


@pytest.mark.parametrize("B,H,Hk,per_head", [(1, 8, 8, 2552), (4, 32, 16, 2552 + 512), (4, 32, 8, 2552 + 256), (2, 4, 2, 2552 + 1024)])
def test_backward_workspace(B, H, Hk, per_head):
    """Per token and value head at 128 x 128: T and P in three parts, the scalars, two states a chunk; 1 KB a key head."""
    L = 640 if B == 2 else 8192
    for mode in (0, 0x10):
        assert api.infini_attn_gated_delta_backward_workspace_size(B, H, Hk, L, 128, 128, mode) == per_head * B * H * L


def check(name, got, want, live=None):
    if live is not None:
        got, want = torch.where(live, got, 0), torch.where(live, want, 0)
    try:
        near(got, np64(want))
    except AssertionError as e:
        raise AssertionError(f"{name}: {e}") from None
    if got.dtype == FP:
        err = float((got.double() - want).norm() / want.norm())
        assert err <= L2, f"{name}: {err:.2e} in the L2 norm"


def kernels(call):
    """The state kernels that ``call`` launches, as in this file's cases, and what it returns."""
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as p:
        got = call()
        torch.cuda.synchronize()
    found = set()
    for e in p.events():
        m = re.search(r"gd::forward_kernel<[^,]+, \d+, (\d), (\d)>", e.name)
        if m:
            found.add({"0": "o", "2": "s"}[m[2]] + m[1])
        m = re.search(r"gd::both_kernel<[^,]+, \d+, (\d), (?:\(bool\))?(\w+)>", e.name)
        if m:
            found.add(("S" if m[2] in ("1", "true") else "B") + m[1])
    return " ".join(sorted(found)), got


CASES = [  # B, H, Hk, L, dk, dv, lens, kernels of the forward, of the backward
    (2, 20, 10, 130, 128, 128, [130, 67], "o1", "B1"),
    (5, 32, 32, 100, 128, 128, None, "o1", "B1"),
    (4, 25, 25, 130, 33, 50, [130, 1, 64, 0], "o1", "B1"),
    (3, 50, 25, 150, 64, 128, None, "o1", "B1"),
    (1, 6, 3, 5000, 128, 128, None, "o1 s1", "B4"),
    (1, 3, 1, 5000, 128, 128, [4321], "o4 s4", "B1 S1"),
    (1, 5, 5, 6000, 64, 128, None, "o1 s1", "B1 S1"),
    (4, 1, 1, 5000, 128, 128, [5000, 0, 64, 2100], "o4 s1", "B1 S1"),
    (1, 8, 4, 5000, 64, 64, None, "o4 s1", "B1 S1"),
    (1, 3, 3, 3000, 128, 48, None, "o4 s4", "B4 S1"),
    (2, 2, 1, 4000, 33, 128, [1, 4000], "o4 s4", "B1 S1"),
    (2, 3, 3, 2000, 64, 16, [2000, 1999], "o4", "B4 S1"),
    (1, 1, 1, 2500, 128, 128, None, "o4 s4", "B4 S4"),
]


@gpu
@types
@pytest.mark.parametrize("B,H,Hk,L,dk,dv,lens,fwd,bwd", CASES)
def test_state_kernels(B, H, Hk, L, dk, dv, lens, fwd, bwd, t):
    x, d_out, dS = backward_inputs(B, H, Hk, L, dk, dv, t, seed=41)
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    o, S, grads = reference(x, dk ** -0.5, n, d_out, dS)
    ran, got = kernels(lambda: forward(*x, lens=n))
    assert ran == fwd
    live = ~torch.isnan(o)
    check("out", got[0], o, live)
    assert bool((got[0][~live] == 7.0).all())
    check("S", got[1], S)
    ran, got = kernels(lambda: api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS, lens=n))
    assert ran == bwd
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, grads):
        check(name, a, w)


@gpu
@types
@pytest.mark.parametrize("H,kernels_of", [(8, "4"), (40, "1")])
def test_long_memories(H, kernels_of, t):
    """Hardly any decay and few key rows, whose writes replace each other: every operand's low parts reach the state."""
    x = make(1, H, H, 640, 16, 128, t, seed=44, decay=0.002)
    _, d_out, dS = backward_inputs(1, H, H, 640, 16, 128, t, seed=44)
    o, S, grads = reference(x, 0.25, None, d_out, dS)
    ran, got = kernels(lambda: forward(*x))
    assert ran == "o" + kernels_of
    check("out", got[0], o)
    check("S", got[1], S)
    ran, got = kernels(lambda: api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS))
    assert ran == "B" + kernels_of
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, grads):
        check(name, a, w)


@gpu
def test_scalar_gradients_of_bf16_inputs():
    """dg and dbeta are fp32 whatever the inputs' type.  They come from sums of 16 terms a step over 128 rows: 8 additions,
    each truncating by 2^-24 of the sum in the mean, 8 * 2^-24 = 2^-21 if all have one sign.  (With the products of the
    operands' low parts in the same sums it is 24 additions.)"""
    x, d_out, dS = backward_inputs(1, 8, 8, 1024, 128, 128, BF, seed=45)
    grads = reference(x, 128 ** -0.5, None, d_out, dS)[2]
    got = api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS)
    for a, w in zip(got[3:5], grads[3:5]):
        assert float((a.double() - w).norm() / w.norm()) <= 2.0 ** -21


@gpu
@pytest.mark.parametrize("H,L", [(8, 1024), (40, 130)])
def test_results_of_fp32_inputs(H, L):
    """The bound of test_scalar_gradients_of_bf16_inputs for what comes from inputs of 24 bits; dk, the sum of four
    products one after the other, twice that."""
    x, d_out, dS = backward_inputs(1, H, H, L, 128, 128, FP, seed=46)
    o, S, grads = reference(x, 128 ** -0.5, None, d_out, dS)
    got = (*forward(*x), *api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS))
    for name, a, w in zip(("out", "S", "dq", "dk", "dv", "dg", "dbeta", "dS0"), got, (o, S, *grads)):
        err = float((a.double() - w).norm() / w.norm())
        assert err <= 2.0 ** (-20 if name == "dk" else -21), f"{name}: {err:.2e}"


@gpu
@types
@pytest.mark.parametrize("g", [-6.0, -15.0, -30.0])
def test_gradient_of_strong_decays(g, t):
    """dg is e^g of what the other gradients are, and as near, by its own size."""
    x, d_out, dS = backward_inputs(2, 4, 2, 150, 64, 48, t, seed=47)
    x[3][:] = g * (1 + 0.1 * torch.rand(x[3].shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV))
    grads = reference(x, 0.125, None, d_out, dS)[2]
    got = api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS)
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, grads):
        check(name, a, w)


@gpu
def test_slabs_of_segments():
    """More chunks than the workspace holds at once, of few enough heads that every slab is cut into segments."""
    B, H, L, dk, dv = 1, 40, 130000, 16, 16
    x = make(B, H, 20, L, dk, dv, decay=0.02, seed=42)
    o, S = reference(x, dk ** -0.5)
    for t in (BF, FP):
        one = api.infini_attn_gated_delta_workspace_size(B, H, 20, 65000, dk, dv, 0x10 if t == FP else 0)
        assert api.infini_attn_gated_delta_workspace_size(B, H, 20, L, dk, dv, 0x10 if t == FP else 0) < 1.5 * one
        y = [z.to(t) for z in x[:3]]
        ran, got = kernels(lambda: forward(*y, *x[3:]))
        assert ran == ("o1 o4 s1" if t == BF else "o4 s1")  # the last slab is shorter
        check("out", got[0], o)
        check("S", got[1], S)


@gpu
def test_a_million_tokens_in_one_call_and_in_pieces():
    """1,048,576 tokens of eight heads, several slabs of several segments each: the same as pieces of one slab."""
    L, piece = 1 << 20, 1 << 17
    q, k, v, g, beta, S0 = make(1, 8, 8, L, 128, 128, decay=0.02, seed=43)
    ran, (out, S) = kernels(lambda: forward(q, k, v, g, beta, S0))
    assert ran == "o1 o4 s1 s4"  # the last slab is shorter
    for i in range(0, L, piece):
        o, S0 = forward(*(y[:, :, i:i + piece] for y in (q, k, v, g, beta)), S0)
        part = out[:, :, i:i + piece].float()
        # two roundings to bf16, and what is within the bounds of an fp32 result on either side
        assert float((part - o.float()).abs().max()) <= 2.0 ** -7 * float(o.abs().max())
        assert float((part - o.float()).norm() / o.float().norm()) <= 2.0 ** -8
    assert float((S - S0).norm() / S0.norm()) <= 2 * L2
