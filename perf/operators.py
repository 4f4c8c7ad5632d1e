"""Cases for the gated delta rule and layer normalisation: what they are given, their plain form and their exact values.

Gated delta rule, per (batch row, value head), with a state S [dk, dv], a log decay g and a write strength beta per token:

    S' = exp(g_t) S_{t-1},  u_t = beta_t (v_t - S'^T k_t),  S_t = S' + k_t u_t^T,  o_t = scale S_t^T q_t

Value head h reads key head h // (H / Hk).  "forward" takes a whole sequence, "step" one token of every request (the
state of request b in row slots[b] of a pool; a negative slot is a padded request), "backward" the gradients of a
sequence.  Rows of a batch entry at and past lens[b] are padding: they leave outputs and state as they were, and their
gradients are 0.

Layer normalisation of the last dimension: y = (x - mean) / sqrt(var + eps) * weight + bias, and its gradients.
"""

import math

import torch

own = False

DEV = "cuda"
CHUNK = 64
EPS = 1e-5


def listed():
    gd = dict(dk=128, dv=128, dtype="bf16", lens=False, state_grad=True)
    return [
        # a long document through one layer of the 1B shape (prefill)
        dict(gd, name="gd_forward_1b", op="forward", B=1, H=8, Hk=8, L=32768),
        # a padded batch of prompts, two value heads to a key head
        dict(gd, name="gd_forward_batch", op="forward", B=4, H=32, Hk=16, L=4096, lens=True),
        # a short odd prompt in fp32 with small heads
        dict(gd, name="gd_forward_fp32_odd", op="forward", B=3, H=6, Hk=3, L=77, dk=48, dv=80, dtype="fp32"),
        # one request being decoded: latency
        dict(gd, name="gd_step_one", op="step", B=1, H=8, Hk=8, L=1),
        # a full serving batch, some of its slots padding
        dict(gd, name="gd_step_batch", op="step", B=192, H=32, Hk=16, L=1, lens=True),
        # training on one long sequence of the 1B shape
        dict(gd, name="gd_backward_1b", op="backward", B=1, H=8, Hk=8, L=32768, state_grad=False),
        # training on a padded batch with shared key heads, resumed from a state
        dict(gd, name="gd_backward_shared", op="backward", B=2, H=16, Hk=8, L=1000, lens=True),
        # a small odd fp32 problem
        dict(gd, name="gd_backward_fp32_odd", op="backward", B=2, H=4, Hk=2, L=150, dk=40, dv=64, dtype="fp32"),
        # a few tokens of a serving step, and a training batch's tokens
        dict(name="ln_forward_tokens", op="ln_forward", rows=8, D=1024, dtype="bf16", wtype="bf16", bias=True),
        dict(name="ln_forward_wide", op="ln_forward", rows=32768, D=4096, dtype="bf16", wtype="fp32", bias=True),
        # the gradients of a training batch, and of odd rows without a bias
        dict(name="ln_backward_1b", op="ln_backward", rows=32768, D=1024, dtype="bf16", wtype="fp32", bias=True),
        dict(name="ln_backward_odd", op="ln_backward", rows=1013, D=1500, dtype="fp32", wtype="fp32", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "step", "backward", "ln_forward", "ln_backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op.startswith("ln"):
        D = _log(rng, 64, 8192)
        rows = _log(rng, 1, max(1, min(262144, (32768 * (4096 if op == "ln_forward" else 1024)) // D)))
        return dict(op=op, rows=rows, D=D, dtype=dtype, wtype=rng.choice([dtype, "fp32"]), bias=rng.random() < 0.7)
    group = rng.choice([1, 1, 2, 4])
    Hk = _log(rng, 1, 16)
    H = Hk * group
    if rng.random() < 0.6:
        dk = dv = 128
    else:
        dk, dv = rng.choice([16, 33, 64, 96, 128]), rng.choice([16, 50, 64, 100, 128])
    B = _log(rng, 1, 8)
    if op == "step":
        B, L = _log(rng, 1, 192 * 32 // H), 1
    else:
        most = 32768 * 8 // (B * H) if op == "backward" or dtype == "fp32" else 4 * 32 * 4096 // (B * H)
        L = _log(rng, 1, max(2, min(16384, most)))
    return dict(op=op, B=B, H=H, Hk=Hk, L=L, dk=dk, dv=dv, dtype=dtype, lens=rng.random() < 0.4,
                state_grad=rng.random() < 0.5)


def _type(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    t = _type(case["dtype"])

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if case["op"].startswith("ln"):
        rows, D = case["rows"], case["D"]
        wt = _type(case["wtype"])
        # residual-stream rows: each with a mean and a size of its own
        x = (randn(rows, D) * torch.exp(0.5 * randn(rows, 1)) + 0.3 * randn(rows, 1)).to(t)
        st = dict(case=case, x=x, weight=(1 + 0.2 * randn(D)).to(wt), bias=(0.2 * randn(D)).to(wt) if case["bias"] else None)
        if case["op"] == "ln_forward":
            st["y"] = torch.empty_like(x)
        else:
            st["d_y"] = randn(rows, D).to(t)
        return st

    B, H, Hk, L, dk, dv = (case[n] for n in ("B", "H", "Hk", "L", "dk", "dv"))
    q = torch.nn.functional.normalize(randn(B, Hk, L, dk), dim=-1).to(t)
    k = torch.nn.functional.normalize(randn(B, Hk, L, dk), dim=-1).to(t)
    v = randn(B, H, L, dv).to(t)
    beta = torch.sigmoid(randn(B, H, L))
    # decay: a rate in [1, 16] per head times a step size around [0.001, 0.1], input dependent
    rate = 1 + 15 * torch.rand(1, H, 1, generator=gen, device=DEV)
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(1, H, 1, generator=gen, device=DEV))
    g = -rate * torch.nn.functional.softplus(torch.log(torch.expm1(step)) + 0.5 * randn(B, H, L))
    st = dict(case=case, q=q, k=k, v=v, g=g.contiguous(), beta=beta, lens=None, slots=None)
    if case["op"] == "step":
        pool = B
        for n in ("q", "k", "v", "g", "beta"):
            st[n] = st[n][:, :, 0].contiguous()
        if case["lens"]:  # requests own scattered rows of a larger pool; about one in sixteen is padding
            pool = B + max(1, B // 4)
            perm = torch.randperm(pool, generator=gen, device=DEV)[:B].to(torch.int32)
            pad = torch.rand(B, generator=gen, device=DEV) < 1 / 16
            st["slots"] = torch.where(pad, torch.full_like(perm, -1), perm)
        st["S"] = 0.3 * randn(pool, H, dk, dv)
        st["out"] = torch.zeros(B, H, dv, dtype=t, device=DEV)
        return st
    if case["lens"]:
        st["lens"] = torch.randint(0, L + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
        st["lens"][0] = L
    S0 = 0.3 * randn(B, H, dk, dv)
    if case["op"] == "forward":
        st["S"], st["out"] = S0, torch.zeros(B, H, L, dv, dtype=t, device=DEV)
    else:
        st["d_out"] = randn(B, H, L, dv).to(t)
        st["S0"], st["dS"] = (S0, 0.1 * randn(B, H, dk, dv)) if case["state_grad"] else (None, None)
    return st


# ---------------------------------------------------------------- plain form


def _chunked(q, k, v, g, beta, S, scale):
    """The recurrence over chunks of 64 tokens in fp32 (decays summed in 64 bits): inside a chunk the writes u solve a
    unit lower triangular system, whose inverse is the product of (I + X^(2^i)) for the nilpotent X = -A."""
    B, H, L, dk = q.shape
    dv = v.shape[3]
    n = -(-L // CHUNK)
    pad = n * CHUNK - L

    def cut(x):
        x = torch.cat([x, x.new_zeros(B, H, pad, *x.shape[3:])], 2) if pad else x
        return x.reshape(B, H, n, CHUNK, *x.shape[3:])

    q, k, v, g, beta = cut(q), cut(k), cut(v), cut(g), cut(beta)
    G = g.double().cumsum(-1)
    eye = torch.eye(CHUNK, device=q.device)
    low = torch.ones(CHUNK, CHUNK, device=q.device).tril()
    diff = (G[..., :, None] - G[..., None, :]).float()
    D = torch.exp(torch.where(low > 0, diff, diff.new_full((), -math.inf)))
    X = -(beta[..., None] * (k @ k.transpose(-1, -2)) * D * (1 - eye))
    T = eye + X
    for _ in range(5):
        X = X @ X
        T = T @ (eye + X)
    P = scale * (q @ k.transpose(-1, -2)) * D
    into = torch.exp(G).float()[..., None]
    rest = torch.exp(G[..., -1:] - G).float()[..., None]
    full = torch.exp(G[..., -1]).float()[..., None, None]
    W, U0 = T @ (beta[..., None] * into * k), T @ (beta[..., None] * v)
    qs, ks = scale * into * q, (rest * k).transpose(-1, -2)
    outs = []
    for c in range(n):  # the state passes from chunk to chunk
        U = U0[:, :, c] - W[:, :, c] @ S
        outs.append(qs[:, :, c] @ S + P[:, :, c] @ U)
        S = full[:, :, c] * S + ks[:, :, c] @ U
    return torch.stack(outs, 2).reshape(B, H, n * CHUNK, dv)[:, :, :L], S


def _valid(lens, B, L):
    """[B, 1, L, 1] truth values of the tokens that are not padding."""
    at = torch.arange(L, device=DEV)
    return (at[None, :] < lens.long()[:, None])[:, None, :, None] if lens is not None else None


def _masked(q, k, v, g, beta, lens, group):
    """fp32 inputs, key heads repeated; a padded token neither decays nor writes."""
    q, k = (x.float().repeat_interleave(group, 1) if group > 1 else x.float() for x in (q, k))
    v = v.float()
    ok = _valid(lens, q.shape[0], q.shape[2])
    if ok is None:
        return q, k, v, g, beta
    return q * ok, k * ok, v * ok, g * ok[..., 0], beta * ok[..., 0]


def _plain_forward(st):
    c = st["case"]
    o, S = _chunked(*_masked(st["q"], st["k"], st["v"], st["g"], st["beta"], st["lens"], c["H"] // c["Hk"]), st["S"],
                    c["dk"] ** -0.5)
    o = o.to(st["out"].dtype)
    ok = _valid(st["lens"], c["B"], c["L"])
    st["out"].copy_(o if ok is None else torch.where(ok, o, st["out"]))
    st["S"].copy_(S)
    return st["out"], st["S"]


def _plain_step(st):
    c = st["case"]
    group, t = c["H"] // c["Hk"], st["out"].dtype
    q, k = (st[n].float().repeat_interleave(group, 1) for n in ("q", "k"))
    at = torch.arange(c["B"], device=DEV) if st["slots"] is None else st["slots"].long()
    ok = (at >= 0)[:, None, None]
    row = at.clamp(min=0)
    S = st["S"][row] * torch.exp(st["g"])[..., None, None]
    u = st["beta"][..., None] * (st["v"].float() - (S * k[..., None]).sum(2))
    S = S + k[..., None] * u[:, :, None]
    o = c["dk"] ** -0.5 * (S * q[..., None]).sum(2)
    if st["slots"] is None:
        st["S"].copy_(S)
    else:
        st["S"].index_copy_(0, at[at >= 0], S[at >= 0])
    st["out"].copy_(torch.where(ok, o.to(t), st["out"]))
    return st["out"], st["S"]


def _plain_backward(st):
    c = st["case"]
    leaves = [st[n].detach().float().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    S0 = st["S0"] if st["S0"] is not None else torch.zeros(c["B"], c["H"], c["dk"], c["dv"], device=DEV)
    S0 = S0.detach().requires_grad_()
    d_out = st["d_out"].float()
    ok = _valid(st["lens"], c["B"], c["L"])
    with torch.enable_grad():
        o, S = _chunked(*_masked(*leaves, st["lens"], c["H"] // c["Hk"]), S0, c["dk"] ** -0.5)
        outs, seeds = [o], [d_out if ok is None else d_out * ok]
        if st["dS"] is not None:
            outs, seeds = outs + [S], seeds + [st["dS"]]
        grads = torch.autograd.grad(outs, leaves + [S0], seeds)
    t = st["q"].dtype
    dq, dk, dv, dg, dbeta, dS0 = grads
    return dq.to(t), dk.to(t), dv.to(t), dg, dbeta, dS0 if c["state_grad"] else None


def _norm(x):
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    return d * rstd, rstd


def _plain_ln_forward(st):
    xhat, _ = _norm(st["x"].float())
    y = xhat * st["weight"].float()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    st["y"].copy_(y.to(st["x"].dtype))
    return st["y"]


def _plain_ln_backward(st):
    xhat, rstd = _norm(st["x"].float())
    dy = st["d_y"].float()
    dxhat = dy * st["weight"].float()
    dx = rstd * (dxhat - dxhat.mean(-1, keepdim=True) - xhat * (dxhat * xhat).mean(-1, keepdim=True))
    t = st["weight"].dtype
    db = dy.sum(0).to(t) if st["bias"] is not None else None
    return dx.to(st["x"].dtype), (dy * xhat).sum(0).to(t), db


# ------------------------------------------------------- the framework's calls


def _own(st):
    from compressive_memory_transformer_sm_b200 import api

    op = st["case"]["op"]
    if op == "forward":
        api.infini_attn_gated_delta_forward(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S"], st["out"],
                                            lens=st["lens"])
        return st["out"], st["S"]
    if op == "step":
        api.infini_attn_gated_delta_step(st["q"], st["k"], st["v"], st["g"], st["beta"], st["S"], st["out"],
                                         slots=st["slots"])
        return st["out"], st["S"]
    if op == "backward":
        return api.infini_attn_gated_delta_backward(st["q"], st["k"], st["v"], st["g"], st["beta"], st["d_out"],
                                                    S0=st["S0"], dS_L=st["dS"], lens=st["lens"],
                                                    want_state_grad=st["case"]["state_grad"])
    if op == "ln_forward":
        api.infini_attn_layer_norm_forward(st["x"], st["weight"], st["bias"], st["y"], eps=EPS)
        return st["y"]
    return api.infini_attn_layer_norm_backward(st["x"], st["weight"], st["d_y"], eps=EPS,
                                               want_bias=st["bias"] is not None)


def run(state):
    if own:
        return _own(state)
    plain = {"forward": _plain_forward, "step": _plain_step, "backward": _plain_backward,
             "ln_forward": _plain_ln_forward, "ln_backward": _plain_ln_backward}
    return plain[state["case"]["op"]](state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("ln"):
        rows, D = case["rows"], case["D"]
        ws = 2 if case["wtype"] == "bf16" else 4
        n = 1 + case["bias"]
        if case["op"] == "ln_forward":
            return {"bytes": 2 * rows * D * es + n * D * ws, "flops": 8 * rows * D}
        return {"bytes": 3 * rows * D * es + (1 + n) * D * ws, "flops": 16 * rows * D}
    B, H, Hk, L, dk, dv = (case[n] for n in ("B", "H", "Hk", "L", "dk", "dv"))
    tok = B * L
    ins = tok * (2 * Hk * dk * es + H * dv * es + 8 * H)
    state = 4 * B * H * dk * dv
    if case["op"] != "backward":
        # S^T k, the write and S^T q
        return {"bytes": ins + tok * H * dv * es + 2 * state, "flops": 6 * tok * H * dk * dv}
    # the recurrence again without its output, S do, dS^T k, dS u, S du and the two rank-one terms of dS
    return {"bytes": 2 * ins + tok * H * dv * es + (3 * state if case["state_grad"] else 0),
            "flops": 16 * tok * H * dk * dv}


# ------------------------------------------------------------------ exact values


def exact(case, seed):
    """64 bits, token by token from the definition."""
    st = prepare(case, seed)
    if case["op"].startswith("ln"):
        return _exact_ln(st)
    f = {n: st[n].double() for n in ("q", "k", "v", "g", "beta")}
    group = case["H"] // case["Hk"]
    scale = 1.0 / math.sqrt(case["dk"])
    if case["op"] == "step":
        return _exact_step(st, f, group, scale)
    B, H, L = case["B"], case["H"], case["L"]
    lens = [L] * B if st["lens"] is None else [int(x) for x in st["lens"].tolist()]
    live = torch.zeros(L, B, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        live[:n, b] = 1
    a = torch.exp(f["g"])
    # [L, B, H, ...]: one contiguous slice per token; a padded token keeps the state (a = 1, beta = 0)
    m = live[:, :, None]
    a = (a.permute(2, 0, 1) * m + (1 - m)).contiguous()
    beta = (f["beta"].permute(2, 0, 1) * m).contiguous()

    def rows(x, heads):
        x = x.permute(2, 0, 1, 3)
        return (x if heads == H else x[:, :, torch.arange(H, device=DEV) // group]).contiguous()

    q, k, v = rows(f["q"], case["Hk"]), rows(f["k"], case["Hk"]), rows(f["v"], H)
    if case["op"] == "forward":
        S = st["S"].double()
        out = st["out"].double()
        for t in range(L):
            S = S * a[t][..., None, None]
            u = beta[t][..., None] * (v[t] - torch.matmul(k[t][..., None, :], S)[..., 0, :])
            S = torch.baddbmm(S.flatten(0, 1), k[t].flatten(0, 1)[..., None], u.flatten(0, 1)[:, None]).view_as(S)
            out[:, :, t] = scale * torch.matmul(q[t][..., None, :], S)[..., 0, :]
        for b, n in enumerate(lens):
            out[b, :, n:] = st["out"][b, :, n:].double()
        return out, S
    return _exact_backward(st, q, k, v, a, beta, live, scale, group)


def _exact_step(st, f, group, scale):
    S, out = st["S"].double(), st["out"].double()
    c = st["case"]
    slots = range(c["B"]) if st["slots"] is None else st["slots"].tolist()
    head = torch.arange(c["H"], device=DEV) // group
    for b, s in enumerate(slots):
        if s < 0:
            continue
        M = S[s] * torch.exp(f["g"][b])[:, None, None]
        kb, qb = f["k"][b][head], f["q"][b][head]
        u = f["beta"][b][:, None] * (f["v"][b] - torch.einsum("hk,hkv->hv", kb, M))
        M = M + torch.einsum("hk,hv->hkv", kb, u)
        S[s] = M
        out[b] = scale * torch.einsum("hk,hkv->hv", qb, M)
    return out, S


def _exact_backward(st, q, k, v, a, beta, live, scale, group):
    c = st["case"]
    B, H, Hk, L, dk, dv = (c[n] for n in ("B", "H", "Hk", "L", "dk", "dv"))
    d_out = (st["d_out"].double() * live.t()[:, None, :, None]).permute(2, 0, 1, 3).contiguous()
    S = st["S0"].double() if st["S0"] is not None else torch.zeros(B, H, dk, dv, dtype=torch.float64, device=DEV)
    every, kept = 128, []

    def forward(S, t):
        S = S * a[t][..., None, None]
        u = beta[t][..., None] * (v[t] - torch.matmul(k[t][..., None, :], S)[..., 0, :])
        return S, u, S + k[t][..., :, None] * u[..., None, :]

    for t in range(L):
        if t % every == 0:
            kept.append(S)
        S = forward(S, t)[2]
    dS = st["dS"].double() if st["dS"] is not None else torch.zeros_like(S)
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(a), torch.zeros_like(beta)
    for n in reversed(range(len(kept))):
        S, hist = kept[n], []
        for t in range(n * every, min(L, (n + 1) * every)):
            Sd, u, S2 = forward(S, t)
            hist.append((t, S, Sd, u, S2))
            S = S2
        for t, Sp, Sd, u, S2 in reversed(hist):
            do = d_out[t][..., None, :]
            dq[t] = scale * (S2 * do).sum(-1)
            dS = dS + scale * q[t][..., :, None] * do
            du = torch.matmul(k[t][..., None, :], dS)
            e = v[t] - torch.matmul(k[t][..., None, :], Sd)[..., 0, :]
            db[t] = (du[..., 0, :] * e).sum(-1)
            dvv[t] = beta[t][..., None] * du[..., 0, :]
            dkk[t] = (dS * u[..., None, :]).sum(-1) - (Sd * dvv[t][..., None, :]).sum(-1)
            dS = dS - k[t][..., :, None] * dvv[t][..., None, :]
            dg[t] = a[t] * (dS * Sp).sum((-1, -2))
            dS = dS * a[t][..., None, None]
    dg, db = dg * live[:, :, None], db * live[:, :, None]

    def back(x):
        x = (x * live[:, :, None, None]).permute(1, 2, 0, 3)
        return x

    def shared(x):
        return back(x).reshape(B, Hk, group, L, dk).sum(2)

    return (shared(dq), shared(dkk), back(dvv), dg.permute(1, 2, 0), db.permute(1, 2, 0),
            dS if c["state_grad"] else None)


def _exact_ln(st):
    x, w = st["x"].double(), st["weight"].double()
    D = x.shape[1]
    mu = x.sum(1, keepdim=True) / D
    var = (x * x).sum(1, keepdim=True) / D - mu * mu
    sd = torch.sqrt(var + EPS)
    z = (x - mu) / sd
    if st["case"]["op"] == "ln_forward":
        return z * w + (st["bias"].double() if st["bias"] is not None else 0.0)
    dy = st["d_y"].double()
    h = dy * w
    dx = (h - h.sum(1, keepdim=True) / D - z * ((h * z).sum(1, keepdim=True) / D)) / sd
    return dx, torch.einsum("rd,rd->d", dy, z), dy.sum(0) if st["bias"] is not None else None
