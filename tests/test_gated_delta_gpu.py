"""The gated delta rule's calls against the fp64 oracle.

Tolerances.  u = 2^-24.  A product of the recurrence sums at most dk (or, inside a chunk, 64) terms: its error is at
most (dk + 64) u of the sum of their magnitudes, which is at most a small multiple of the result's largest magnitude
for the keys used here (unit length) -- taken as 4.  What earlier tokens left is contracted by every later one (decay
at most 1, beta |k|^2 <= 2), so that it adds no more than the last steps do: 4 * 192 u = 4.6e-5 of the largest
magnitude, elementwise, for every fp32 result.  A bf16 result adds half a step, 2^-8 of its value."""

import numpy as np
import pytest
import torch

from compressive_memory_transformer_sm_b200 import api
from oracle import gated_delta as G

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 4 * 192 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, FP = torch.bfloat16, torch.float32


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def near(got, want, where=None):
    a, w = np64(got), want
    assert a.shape == w.shape
    bound = TOL * np.abs(np.where(np.isnan(w), 0, w)).max() + HALF[got.dtype] * np.abs(w) * 1.01
    ok = np.abs(a - w) <= bound
    ok = ok if where is None else ok | ~where
    assert ok.all(), f"{(~ok).sum()} of {ok.size} off, worst {np.nanmax(np.where(ok, 0, np.abs(a - w))):.3e}, size {np.nanmax(np.abs(w)):.3e}"


def make(B, H, Hk, L, dk, dv, t=BF, seed=0, decay=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed + 7919 * L + dk)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(x, dim=-1)  # noqa: E731
    q, k = unit(r(B, Hk, L, dk)).to(t), unit(r(B, Hk, L, dk)).to(t)
    v = r(B, H, L, dv).to(t)
    g = -decay * torch.nn.functional.softplus(r(B, H, L) - 2)
    beta = torch.sigmoid(r(B, H, L))
    return q, k, v, g, beta, 0.3 * r(B, H, dk, dv)


def forward(q, k, v, g, beta, S0, scale=0.0, lens=None, **kw):
    S, out = S0.clone(), torch.full_like(v, 7.0)
    api.infini_attn_gated_delta_forward(q, k, v, g, beta, S, out, scale=scale, lens=lens, **kw)
    return out, S


def check_forward(q, k, v, g, beta, S0, out, S, scale=0.0, lens=None):
    n = None if lens is None else lens.tolist()
    wo, wS = G.forward(*map(np64, (q, k, v, g, beta, S0)), scale or q.shape[-1] ** -0.5, n)
    live = ~np.isnan(wo)
    near(out, np.where(live, wo, 0), live)
    assert bool((out[torch.from_numpy(~live).to(DEV)] == 7.0).all())  # rows behind the end stay as they were
    near(S, wS)


SHAPES = [  # B, H, Hk, L, dk, dv
    (1, 1, 1, 1, 128, 128), (2, 2, 1, 3, 16, 16), (1, 3, 3, 63, 128, 128), (1, 2, 2, 64, 64, 64), (1, 2, 1, 65, 128, 64),
    (2, 4, 2, 130, 33, 50), (2, 8, 8, 19, 128, 128), (1, 2, 2, 20, 128, 64), (1, 2, 1, 36, 64, 128), (1, 2, 2, 200, 96, 100), (1, 1, 1, 257, 128, 128), (1, 4, 1, 129, 1, 1), (1, 2, 2, 100, 7, 128),
    (1, 2, 1, 77, 128, 3), (1, 1, 1, 1100, 128, 128),
]


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,L,dk,dv", SHAPES)
def test_forward(B, H, Hk, L, dk, dv, t):
    x = make(B, H, Hk, L, dk, dv, t)
    check_forward(*x, *forward(*x))


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
def test_forward_lens(t):
    x = make(6, 4, 2, 200, 128, 96, t)
    lens = torch.tensor([0, 1, 64, 199, 300, -5], dtype=torch.int32, device=DEV)
    q, k, v, g, beta, S0 = x
    for b, n in enumerate(lens.tolist()):  # what lies behind a row's end is not read
        n = min(max(n, 0), 200)
        for y in (q, k, v, g, beta):
            y[b, :, n:] = float("nan")
    out, S = forward(*x, lens=lens)
    clean = [torch.nan_to_num(y) for y in x]
    check_forward(*clean, out, S, lens=lens)
    assert torch.equal(S[0], S0[0]) and torch.equal(S[5], S0[5])


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
def test_forward_strides_and_scale(t):
    """Heads packed beside each other per token, odd strides, and one tensor broadcast over the heads."""
    B, H, L, dk, dv = 2, 3, 150, 40, 24
    q, k, v, g, beta, S0 = make(B, H, H, L, dk, dv, t)
    packed = torch.cat([x.transpose(1, 2).reshape(B, L, -1) for x in (q, k, v)], -1)
    q2, k2, v2 = packed.split([H * dk, H * dk, H * dv], -1)
    q2, k2, v2 = (x.view(B, L, H, -1).transpose(1, 2) for x in (q2, k2, v2))
    g2 = g.transpose(1, 2).contiguous().transpose(1, 2)
    b2 = beta[:, :1].expand(B, H, L)
    out = torch.full((B, L, H, dv + 1), 7.0, dtype=t, device=DEV)[..., :dv].transpose(1, 2)
    S = S0.clone()
    api.infini_attn_gated_delta_forward(q2, k2, v2, g2, b2, S, out, scale=0.5)
    check_forward(q, k, v, g, b2, S0, out, S, scale=0.5)


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
def test_decays(t):
    """No decay at all, decays that leave nothing, and tokens that clear the state."""
    q, k, v, g, beta, S0 = make(1, 4, 4, 160, 64, 32, t)
    g[:, 0] = 0
    g[:, 1] = -40.0
    g[:, 2, ::9] = float("-inf")
    g[:, 3, 70:] = -1e30
    beta[:, 3, 3:9] = 0
    beta[:, 0, 5:60] = 2.0
    x = (q, k, v, g, beta, S0)
    check_forward(*x, *forward(*x))


def test_equal_keys():
    """Every key the same: the chunk's triangular system has no small entries."""
    q, k, v, g, beta, S0 = make(1, 2, 2, 192, 128, 128)
    k[:] = k[:, :, :1]
    beta[:, 0] = 1.0
    x = (q, k, v, g, beta, S0)
    check_forward(*x, *forward(*x))


@pytest.mark.parametrize("L,cut", [(300, 100), (300, 256), (1024, 1023)])
def test_forward_in_pieces_and_steps(L, cut):
    """A sequence, its two pieces, and its prefill followed by single tokens give the same results."""
    x = make(2, 4, 2, L, 128, 128, seed=3)
    q, k, v, g, beta, S0 = x
    out, S = forward(*x)
    first = [y[:, :, :cut] for y in x[:5]]
    o1, S1 = forward(*first, S0)
    size = float(out.abs().max())
    assert float((o1.float() - out[:, :, :cut].float()).abs().max()) <= (TOL + 2 ** -7) * size
    rest = [y[:, :, cut:] for y in x[:5]]
    o2, S2 = forward(*rest, S1)
    near(S2, np64(S))
    assert float((o2.float() - out[:, :, cut:].float()).abs().max()) <= (TOL + 2 ** -7) * size
    S3, o3 = S1.clone(), torch.empty(2, 4, 128, dtype=BF, device=DEV)
    for i in range(cut, min(L, cut + 50)):
        api.infini_attn_gated_delta_step(q[:, :, i], k[:, :, i], v[:, :, i], g[:, :, i], beta[:, :, i], S3, o3)
        assert float((o3.float() - out[:, :, i].float()).abs().max()) <= (TOL + 2 ** -7) * size
    if L - cut <= 50:
        near(S3, np64(S))


def test_repeats_bit_for_bit_and_rows_are_independent():
    x = make(3, 4, 2, 500, 128, 128, seed=5)
    out, S = forward(*x)
    again = forward(*x)
    assert torch.equal(out, again[0]) and torch.equal(S, again[1])
    one = forward(*[y[1:2].contiguous() for y in x])
    near(one[1], np64(S[1:2]))


STEPS = [(1, 8, 8, 128, 128, BF), (5, 4, 2, 128, 128, BF), (3, 6, 3, 48, 80, FP), (2, 2, 1, 33, 50, BF), (1, 1, 1, 1, 1, FP),
         (40, 8, 2, 64, 100, BF), (2, 3, 1, 16, 18, FP)]


def check_step(q, k, v, g, beta, S0, out, S, slots):
    for b in range(q.shape[0]):
        s = b if slots is None else slots[b]
        if not 0 <= s < S0.shape[0]:
            assert bool((out[b] == 7.0).all())
            continue
        wo, wS = G.forward(*[np64(y[b:b + 1])[:, :, None] for y in (q, k, v, g, beta)], np64(S0[s:s + 1]),
                           q.shape[-1] ** -0.5)
        near(out[b:b + 1], wo[:, :, 0])
        near(S[s:s + 1], wS)
    for s in range(S0.shape[0]):
        if slots is not None and s not in slots:
            assert torch.equal(S[s], S0[s])


@pytest.mark.parametrize("B,H,Hk,dk,dv,t", STEPS)
def test_step(B, H, Hk, dk, dv, t):
    q, k, v, g, beta, _ = (y[:, :, 0] if y.dim() < 5 else y for y in make(B, H, Hk, 1, dk, dv, t))
    S0 = torch.randn(B + 3, H, dk, dv, device=DEV)
    order = torch.randperm(B + 3)[:B].tolist()
    order[B // 2] = -1 if B > 1 else order[0]
    if B > 2:
        order[-1] = B + 3
    for slots in (None, order):
        S, out = S0.clone(), torch.full((B, H, dv), 7.0, dtype=t, device=DEV)
        sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device=DEV)
        api.infini_attn_gated_delta_step(q, k, v, g, beta, S, out, slots=sl)
        check_step(q, k, v, g, beta, S0, out, S, slots)


def test_step_same_slot_in_order():
    """Requests that name one slot are one sequence."""
    q, k, v, g, beta, S0 = make(1, 4, 2, 5, 128, 64)
    want_o, want_S = G.forward(*map(np64, (q, k, v, g, beta, S0)), 128 ** -0.5)
    rows = [y[0].transpose(0, 1).contiguous() for y in (q, k, v, g, beta)]
    pad = [torch.cat([y, y[:1]]) for y in rows]
    S, out = torch.cat([torch.zeros_like(S0), S0]), torch.full((6, 4, 64), 7.0, dtype=BF, device=DEV)
    api.infini_attn_gated_delta_step(*pad, S, out, slots=torch.tensor([1, 1, 1, 1, 1, -1], dtype=torch.int32, device=DEV))
    near(S[1:], want_S)
    near(out[:5], want_o[0].transpose(1, 0, 2))
    assert bool((out[5] == 7.0).all()) and not S[0].any()


def test_streams_workspaces_and_graphs():
    x = make(2, 4, 2, 333, 128, 128, seed=11)
    q, k, v, g, beta, S0 = x
    want = forward(*x)
    torch.cuda.synchronize()
    n = api.infini_attn_gated_delta_workspace_size(2, 4, 2, 333, 128, 128)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        S, out = S0.clone(), torch.full_like(v, 7.0)
    api.infini_attn_gated_delta_forward(q, k, v, g, beta, S, out, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(S, want[1])
    # two captured graphs, one on its own workspace and one on the call's, replayed in turn
    graphs, held = [], []
    for space in (ws, None):
        S, out = S0.clone(), torch.full_like(v, 7.0)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            api.infini_attn_gated_delta_forward(q, k, v, g, beta, S, out, workspace=space)
        graphs.append(gr)
        held.append((S, out))
    for S, out in held:
        S.copy_(S0)
        out.fill_(7.0)
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for S, out in held:
        assert torch.equal(out, want[0]) and torch.equal(S, want[1])
    if n:
        with pytest.raises(api.InfiniAttnError):
            api.infini_attn_gated_delta_forward(q, k, v, g, beta, S0.clone(), out, workspace=ws[:n - 256])


def check_backward(x, d_out, dS, got, scale=0.0, lens=None):
    q, k, v, g, beta, S0 = x
    n = None if lens is None else lens.tolist()
    z = torch.zeros(q.shape[0], v.shape[1], q.shape[3], v.shape[3], device=DEV)
    want = G.backward(*map(np64, (q, k, v, g, beta, z if S0 is None else S0, d_out, z if dS is None else dS)),
                      scale or q.shape[-1] ** -0.5, n)
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dS0"), got, want):
        if a is not None:
            try:
                near(a, w)
            except AssertionError as e:
                raise AssertionError(f"{name}: {e}") from None


def backward_inputs(B, H, Hk, L, dk, dv, t, seed=0):
    x = make(B, H, Hk, L, dk, dv, t, seed)
    gen = torch.Generator(device=DEV).manual_seed(seed + 99)
    return x, torch.randn(B, H, L, dv, generator=gen, device=DEV).to(t), 0.3 * torch.randn(B, H, dk, dv, generator=gen, device=DEV)


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,L,dk,dv", [s for s in SHAPES if s[3] < 1000] + [(1, 1, 1, 500, 128, 128)])
def test_backward(B, H, Hk, L, dk, dv, t):
    x, d_out, dS = backward_inputs(B, H, Hk, L, dk, dv, t)
    got = api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS)
    check_backward(x, d_out, dS, got)
    got = api.infini_attn_gated_delta_backward(*x[:5], d_out, want_state_grad=False, scale=0.25)
    assert got[5] is None
    check_backward((*x[:5], None), d_out, None, got, scale=0.25)


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("group", [2, 3])
def test_backward_many_chunks_of_shared_heads(group, t):
    """Enough chunks that one block takes the value heads of a key head in turn."""
    x, d_out, dS = backward_inputs(5, 4 * group, 4, 520, 48, 20, t, seed=group)
    lens = torch.tensor([520, 64, 333, 0, 520], dtype=torch.int32, device=DEV)
    got = api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS, lens=lens)
    check_backward(x, d_out, dS, got, lens=lens)


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
def test_backward_lens(t):
    x, d_out, dS = backward_inputs(6, 4, 2, 200, 128, 48, t)
    lens = torch.tensor([0, 1, 64, 199, 300, -5], dtype=torch.int32, device=DEV)
    dirty = [y.clone() for y in (*x[:5], d_out)]
    for b, n in enumerate(lens.tolist()):
        for y in dirty:
            y[b, :, min(max(n, 0), 200):] = float("nan")
    got = api.infini_attn_gated_delta_backward(*dirty, S0=x[5], dS_L=dS, lens=lens)
    check_backward(x, d_out, dS, got, lens=lens)
    for y in got[:5]:
        for b, n in enumerate(lens.tolist()):
            assert not y[b, :, min(max(n, 0), 200):].any()
    assert torch.equal(got[5][0], dS[0])


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
def test_backward_strides_and_decays(t):
    x, d_out, dS = backward_inputs(2, 3, 1, 150, 40, 24, t, seed=2)
    q, k, v, g, beta, S0 = x
    g[:, 0] = 0
    g[:, 1, ::9] = float("-inf")
    g[:, 2, 70:] = -1e30
    beta[:, 1, 3:9] = 0
    turn = lambda y: y.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    d2 = d_out[:, :1].expand(2, 3, 150, 24)
    got = api.infini_attn_gated_delta_backward(turn(q), turn(k), turn(v), turn(g), turn(beta), d2, S0=S0, dS_L=dS)
    check_backward(x, d2, dS, got)


def test_backward_against_differences():
    """The loss's change along a random direction, from the forward's own fp32 outputs: truncation about eps^2 = 1e-4
    relative and cancellation 2e-6 / 1e-2 = 2e-4 of the loss's terms; 5e-3 holds both."""
    x, d_out, dS = backward_inputs(1, 4, 2, 130, 64, 64, FP, seed=8)
    got = api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS)
    gen = torch.Generator(device=DEV).manual_seed(4)
    for i, (y, dy) in enumerate(zip(x, got)):
        d = torch.randn(y.shape, generator=gen, device=DEV) * y.abs().mean()
        ends = []
        for e in (1e-2, -1e-2):
            z = list(x)
            z[i] = y + e * d
            out, S = forward(*z)
            ends.append(float((out.double() * d_out).sum() + (S.double() * dS).sum()))
        slope, size = (dy.double() * d).sum().item(), (dy.double() * d).norm().item()
        assert abs((ends[0] - ends[1]) / 2e-2 - slope) <= 5e-3 * max(abs(slope), size), i


def test_backward_streams_workspaces_and_graphs():
    x, d_out, dS = backward_inputs(2, 4, 2, 333, 128, 128, BF, seed=12)
    call = lambda **kw: api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS, **kw)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    n = api.infini_attn_gated_delta_backward_workspace_size(2, 4, 2, 333, 128, 128)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    got = call(workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph, held = torch.cuda.CUDAGraph(), None
    with torch.cuda.graph(graph):
        held = call(workspace=ws)
    for _ in range(2):
        for y in held:
            y.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    with pytest.raises(api.InfiniAttnError):
        call(workspace=ws[:n - 256])


def test_norm_memory_and_gradients_together():
    """One layer's pass as a model runs it: norm, q and k of unit length, gated delta rule, and back through both."""
    B, H, L, D = 2, 4, 150, 512
    gen = torch.Generator(device=DEV).manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    x, w, bias = r(B, L, D).to(BF), (1 + 0.1 * r(D)).to(BF), (0.1 * r(D)).to(BF)
    y = torch.empty_like(x)
    api.infini_attn_layer_norm_forward(x, w, bias, y)
    v = y.view(B, L, H, 128).transpose(1, 2)  # the normalised rows are the values, heads side by side
    q, k, _, g, beta, S0 = make(B, H, H, L, 128, 128, seed=4)
    out, S = torch.empty(B, H, L, 128, dtype=BF, device=DEV), S0.clone()
    api.infini_attn_gated_delta_forward(q, k, v, g, beta, S, out)
    d_out = r(B, H, L, 128).to(BF)
    grads = api.infini_attn_gated_delta_backward(q, k, v, g, beta, d_out, S0=S0)
    d_y = grads[2].transpose(1, 2).reshape(B, L, D)
    dx, dw, db = api.infini_attn_layer_norm_backward(x, w, d_y)
    wo, wS = G.forward(*map(np64, (q, k, v, g, beta, S0)), 128 ** -0.5)
    near(out, wo)
    near(S, wS)
    check_backward((q, k, v, g, beta, S0), d_out, None, grads)
    wx, ww, wb = G.layer_norm_backward(*map(np64, (x, w, d_y)), 1e-5)
    near(dx, wx)
    near(dw, ww)
    near(db, wb)


@pytest.mark.parametrize("t", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,L,dk,dv,lens", [(1, 1, 1, 2500, 128, 128, None), (3, 1, 1, 2100, 64, 40, [2100, 0, 700]),
                                                (2, 2, 1, 1700, 33, 128, [1, 1700])])
def test_long_sequences_of_few_heads(B, H, Hk, L, dk, dv, lens, t):
    """Long enough, with few (b, h), for the sequence to be cut into segments that run side by side."""
    x, d_out, dS = backward_inputs(B, H, Hk, L, dk, dv, t, seed=6)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    check_forward(*x, *forward(*x, lens=ln), lens=ln)
    got = api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS, lens=ln)
    check_backward(x, d_out, dS, got, lens=ln)
    got2 = api.infini_attn_gated_delta_backward(*x[:5], d_out, S0=x[5], dS_L=dS, lens=ln)
    assert all(torch.equal(a, b) for a, b in zip(got, got2))


def test_forward_in_slabs():
    """More chunks than the workspace holds at once: the same as row by row, each of which fits."""
    B, H, L = 8, 64, 8192
    q, k, v, g, beta, _ = make(B, H, 8, L, 64, 32, decay=0.1)
    assert api.infini_attn_gated_delta_workspace_size(B, H, 8, L, 64, 32) < api.infini_attn_gated_delta_workspace_size(1, H, 8, L, 64, 32) * B
    lens = torch.tensor([8192, 1, 0, 64, 65, 5000, 8191, 4096], dtype=torch.int32, device=DEV)
    S0 = torch.zeros(B, H, 64, 32, device=DEV)
    out, S = forward(q, k, v, g, beta, S0, lens=lens)
    for b, n in enumerate(lens.tolist()):
        assert bool((out[b, :, n:] == 7.0).all())
        if n:
            o1, S1 = forward(*[y[b:b + 1, :, :n] for y in (q, k, v, g, beta)], S0[b:b + 1])
            near(S[b:b + 1], np64(S1))
            assert float((out[b, :, :n].float() - o1[0].float()).abs().max()) <= (TOL + 2 ** -7) * float(o1.abs().max())


def test_state_pool_past_32_bits():
    pool = 140000  # 2.29e9 elements
    S = torch.empty(pool, 1, 128, 128, device=DEV)
    S[-3:] = 0.1
    q, k, v, g, beta, _ = make(2, 1, 1, 1, 128, 128)
    one = [y[:, :, 0] for y in (q, k, v, g, beta)]
    few, o1, o2 = S[-3:].clone(), torch.zeros(2, 1, 128, dtype=BF, device=DEV), torch.zeros(2, 1, 128, dtype=BF, device=DEV)
    api.infini_attn_gated_delta_step(*one, S, o1, slots=torch.tensor([pool - 1, pool - 3], dtype=torch.int32, device=DEV))
    api.infini_attn_gated_delta_step(*one, few, o2, slots=torch.tensor([2, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(S[-3:], few) and torch.equal(o1, o2)
