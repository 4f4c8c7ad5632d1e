"""Refusals of the gated delta rule's and the layer norm's calls, and their structs' layouts (no kernel is launched)."""

import ctypes

import pytest
import torch

from compressive_memory_transformer_sm_b200 import F32, api

OK = (api.INFINI_OK, api.INFINI_ERR_DEVICE)  # a well-formed call: OK is not reached without a device


def host(n=1 << 16):
    return ctypes.addressof(_BUF) + 256 - ctypes.addressof(_BUF) % 256 + n


_BUF = ctypes.create_string_buffer(1 << 22)


def params(**over):
    p = api.GatedDeltaParams()
    p.q, p.k, p.v, p.g, p.beta, p.S, p.out = (host(i << 18) for i in range(1, 8))
    p.B, p.H, p.Hk, p.L, p.dk, p.dv, p.mode = 1, 2, 1, 4, 16, 8, F32
    for n, x in over.items():
        setattr(p, n, x)
    return p


def step_params(**over):
    p = api.GatedDeltaStepParams()
    p.q, p.k, p.v, p.g, p.beta, p.S, p.out = (host(i << 18) for i in range(1, 8))
    p.B, p.H, p.Hk, p.pool, p.dk, p.dv, p.mode = 2, 2, 1, 4, 16, 8, 0
    for n, x in over.items():
        setattr(p, n, x)
    return p


pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host pointers: refusals only, on machines without a GPU")


def test_struct_sizes():
    for which, cls in enumerate((api.GatedDeltaParams, api.GatedDeltaStepParams, api.GatedDeltaBackwardParams)):
        assert api.lib.infini_attn_gated_delta_params_size(which) == ctypes.sizeof(cls)
    assert api.lib.infini_attn_gated_delta_params_size(7) == 0
    for packed, cls in ((api._GD_FORWARD, api.GatedDeltaParams), (api._GD_STEP, api.GatedDeltaStepParams),
                        (api._GD_BACKWARD, api.GatedDeltaBackwardParams)):
        n = sum(f[1]._length_ if hasattr(f[1], "_length_") else 1 for f in cls._fields_)
        p = cls.from_buffer_copy(packed.pack(*range(1, n + 1)) + bytes(-packed.size % 8))
        flat = []
        for f, _ in cls._fields_:
            x = getattr(p, f)
            flat += list(x) if hasattr(x, "__len__") else [x]
        assert flat == list(range(1, n + 1))


def backward_params(**over):
    p = api.GatedDeltaBackwardParams()
    names = ("q", "k", "v", "g", "beta", "S0", "d_out", "dS_L", "dq", "dk_out", "dv_out", "dg", "dbeta", "dS0")
    for i, n in enumerate(names):
        setattr(p, n, host((i + 1) << 16))
    p.B, p.H, p.Hk, p.L, p.dk, p.dv, p.mode = 1, 2, 1, 4, 16, 8, 0
    for n, x in over.items():
        setattr(p, n, x)
    return p


def backward(**over):
    return api.lib.infini_attn_gated_delta_backward(ctypes.byref(backward_params(**over)))


def forward(**over):
    return api.lib.infini_attn_gated_delta_forward(ctypes.byref(params(**over)))


def step(**over):
    return api.lib.infini_attn_gated_delta_step(ctypes.byref(step_params(**over)))


BAD, UNSUP = api.INFINI_ERR_INVALID_ARG, api.INFINI_ERR_UNSUPPORTED
L3, L2 = ctypes.c_longlong * 3, ctypes.c_longlong * 2


def test_well_formed_calls_reach_the_device_check():
    assert forward() == api.INFINI_ERR_DEVICE and step() == api.INFINI_ERR_DEVICE


@pytest.mark.parametrize("over,rc", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(g=None), BAD), (dict(beta=None), BAD),
    (dict(S=None), BAD), (dict(out=None), BAD), (dict(B=0), BAD), (dict(H=3, Hk=2), BAD), (dict(L=0), BAD),
    (dict(dk=0), BAD), (dict(dv=-1), BAD), (dict(dk=129), UNSUP), (dict(dv=200), UNSUP), (dict(mode=1), UNSUP),
    (dict(L=1 << 32), UNSUP), (dict(q_stride=L3(-16, 0, 16)), BAD), (dict(o_stride=L3(64, 32, 4)), BAD),
    (dict(o_stride=L3(0, 0, 8)), BAD), (dict(B=2, o_stride=L3(8, 0, 16)), BAD),
])
def test_forward_refusals(over, rc):
    assert forward(**over) == rc


def test_overlaps_are_refused():
    p = params()
    assert forward(out=p.v) == BAD and forward(S=p.k) == BAD and forward(out=p.S) == BAD and forward(lens=p.out) == BAD
    s = step_params()
    assert step(out=s.q) == BAD and step(S=s.v) == BAD and step(slots=s.S) == BAD


@pytest.mark.parametrize("over,rc", [
    (dict(S=None), BAD), (dict(B=0), BAD), (dict(H=3, Hk=2), BAD), (dict(pool=0), BAD), (dict(pool=1), BAD),
    (dict(dk=144), UNSUP), (dict(mode=0x20), UNSUP), (dict(pool=1 << 60), UNSUP), (dict(o_stride=L2(8, 8)), BAD),
    (dict(v_stride=L2(-1, 8)), BAD),
])
def test_step_refusals(over, rc):
    assert step(**over) == rc


@pytest.mark.parametrize("over,rc", [
    (dict(), api.INFINI_ERR_DEVICE), (dict(S0=None, dS_L=None, dS0=None), api.INFINI_ERR_DEVICE), (dict(q=None), BAD),
    (dict(d_out=None), BAD), (dict(dq=None), BAD), (dict(dk_out=None), BAD), (dict(dv_out=None), BAD), (dict(dg=None), BAD),
    (dict(dbeta=None), BAD), (dict(H=3, Hk=2), BAD), (dict(L=-1), BAD), (dict(dk=129), UNSUP), (dict(mode=1), UNSUP),
    (dict(d_out_stride=L3(-1, 0, 8)), BAD),
])
def test_backward_refusals(over, rc):
    assert backward(**over) == rc


def test_backward_overlaps_and_workspaces():
    p = backward_params()
    for out in ("dq", "dk_out", "dv_out", "dg", "dbeta", "dS0"):
        assert backward(**{out: p.v}) == BAD and backward(**{out: p.S0}) == BAD
    assert backward(dq=p.dk_out) == BAD and backward(dg=p.dbeta) == BAD and backward(lens=p.dv_out) == BAD
    n = api.infini_attn_gated_delta_backward_workspace_size(1, 2, 1, 4, 16, 8)
    ws = host(20 << 16)
    assert n > 0 and api.infini_attn_gated_delta_backward_workspace_size(1, 3, 2, 4, 16, 8) == 0
    assert backward(workspace=ws, workspace_bytes=n) == api.INFINI_ERR_DEVICE
    assert backward(workspace=ws, workspace_bytes=n - 1) == api.INFINI_ERR_WORKSPACE
    assert backward(workspace=ws + 16, workspace_bytes=n) == api.INFINI_ERR_WORKSPACE
    m = api.infini_attn_gated_delta_workspace_size(1, 2, 1, 100, 16, 8)
    assert m > 0 and api.infini_attn_gated_delta_workspace_size(1, 2, 1, 1, 16, 8) == 0
    assert forward(L=100, workspace=ws, workspace_bytes=m - 1) == api.INFINI_ERR_WORKSPACE


def test_layer_norm_refusals():
    f, b = api.lib.infini_attn_layer_norm_forward, api.lib.infini_attn_layer_norm_backward
    x, w, y, z = (host(i << 18) for i in range(1, 5))
    assert f(x, w, None, y, 4, 32, 1e-5, 0, None) == api.INFINI_ERR_DEVICE
    assert f(x, w, None, x, 4, 32, 1e-5, 0, None) == api.INFINI_ERR_DEVICE
    assert f(None, w, None, y, 4, 32, 1e-5, 0, None) == BAD and f(x, None, None, y, 4, 32, 1e-5, 0, None) == BAD
    assert f(x, w, None, y, 0, 32, 1e-5, 0, None) == BAD and f(x, w, None, y, 4, 0, 1e-5, 0, None) == BAD
    assert f(x, w, None, y, 4, 32, -1.0, 0, None) == BAD and f(x, w, None, y, 4, 32, float("nan"), 0, None) == BAD
    assert f(x, w, None, x + 64, 4, 32, 1e-5, 0, None) == BAD and f(x, w, y, y, 4, 32, 1e-5, 0, None) == BAD
    assert f(x, w, None, y, 4, 16385, 1e-5, 0, None) == UNSUP and f(x, w, None, y, 4, 32, 1e-5, 1, None) == UNSUP
    n = api.infini_attn_layer_norm_backward_workspace_size(4, 32)
    assert n > 0 and api.infini_attn_layer_norm_backward_workspace_size(4, 1 << 20) == 0
    dw, db, ws = (host((8 + i) << 18) for i in range(3))
    assert b(x, w, y, z, dw, db, 4, 32, 1e-5, 0, ws, n, None) == api.INFINI_ERR_DEVICE
    assert b(x, w, y, y, dw, None, 4, 32, 1e-5, 0, ws, n, None) == api.INFINI_ERR_DEVICE
    assert b(x, w, y, z, dw, dw, 4, 32, 1e-5, 0, ws, n, None) == BAD
    assert b(x, w, y, z, w, db, 4, 32, 1e-5, 0, ws, n, None) == BAD
    assert b(x, w, y, z, dw, db, 4, 32, 1e-5, 0, ws, n - 1, None) == api.INFINI_ERR_WORKSPACE
    assert b(x, w, y, z, dw, db, 4, 32, 1e-5, 0, ws + 16, n, None) == api.INFINI_ERR_WORKSPACE


def test_binding_refuses_what_it_cannot_pass_on():
    z = torch.zeros
    q, k, v = z(1, 2, 4, 16), z(1, 2, 4, 16), z(1, 2, 4, 8)
    g, S = z(1, 2, 4), z(1, 2, 16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        api.infini_attn_gated_delta_forward(q, k, v, g, g, S, z(1, 2, 4, 8))
    with pytest.raises(ValueError, match="shape"):
        api.infini_attn_gated_delta_forward(q, k, v, g, g[:, :1], S, z(1, 2, 4, 8))
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        api.infini_attn_gated_delta_forward(q.half(), k, v, g, g, S, v)
    one = torch.tensor(0.0).expand(1, 1, 4)  # one element for four tokens
    with pytest.raises(ValueError, match="broadcast"):
        api.infini_attn_gated_delta_forward(q[:, :1], k[:, :1], v[:, :1], one, g[:, :1], S[:, :1].contiguous(), v[:, :1])
    with pytest.raises(ValueError, match="broadcast"):
        api.infini_attn_gated_delta_forward(q, k, v, torch.tensor(0.0).expand(1, 2, 4), g, S, z(1, 2, 4, 8))
    with pytest.raises(TypeError):
        api.infini_attn_gated_delta_forward(q, None, v, g, g, S, v)
    with pytest.raises(ValueError, match="dimensions"):
        api.infini_attn_gated_delta_step(q, k, v, g, g, S, v)
    with pytest.raises(ValueError, match="shape"):
        api.infini_attn_layer_norm_forward(z(3, 4), z(5), None, z(3, 4))
    with pytest.raises(ValueError, match="must be"):
        api.infini_attn_layer_norm_forward(z(3, 4), z(4), None, z(3, 4, dtype=torch.bfloat16))
