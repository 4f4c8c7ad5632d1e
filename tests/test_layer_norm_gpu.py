"""infini_attn_layer_norm_forward / _backward against the fp64 oracle.

Tolerances, relative to the largest magnitude that enters an element (u = 2^-24, D elements a row):
the sums of a row are trees of at most 16 serial and 15 parallel additions per level, so mean, variance and the two
sums of the backward are within 40 u of their terms' sizes; an element of y or dx is a handful of operations more.
100 u = 6e-6 covers them in fp32 (relative to max |x| / sd * |w|, the size of the terms).  dweight and dbias sum
``rows`` terms: at most rows / grid serial additions, covered by (100 + rows) u times the mean term size * rows,
taken as 2e-6 * sum |terms|.  A bf16 result adds half a step, 2^-8 of its value."""

import numpy as np
import pytest
import torch

from compressive_memory_transformer_sm_b200 import api
from oracle import gated_delta as G

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def np64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def make(rows, D, t, wt, seed, mean=0.5, shift=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731

    def place(x):  # `shift` elements off the allocation's alignment
        flat = torch.empty(x.numel() + shift, dtype=x.dtype, device=DEV)[shift:]
        return flat.view(x.shape).copy_(x)

    x = (r(rows, D) * torch.exp(0.5 * r(rows, 1)) + mean * r(rows, 1)).to(t)
    return place(x), place((1 + 0.2 * r(D)).to(wt)), place((0.2 * r(D)).to(wt)), place(r(rows, D).to(t))


def check_forward(x, w, b, y, eps):
    x64, w64, b64 = np64(x), np64(w), np64(b)
    want = G.layer_norm(x64, w64, b64, eps)
    sd = np.sqrt(x64.var(-1, keepdims=True) + eps)
    size = np.abs(x64).max(-1, keepdims=True) / sd * np.abs(w64) + (0 if b64 is None else np.abs(b64))
    assert np.all(np.abs(np64(y) - want) <= 100 * U * size + HALF[y.dtype] * np.abs(want) * 1.01)


def check_backward(x, w, dy, got, eps, bias=True):
    x64, w64, dy64 = np64(x), np64(w), np64(dy)
    dx, dw, db = G.layer_norm_backward(x64, w64, dy64, eps)
    d = x64 - x64.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    z = np.abs(x64).max(-1, keepdims=True) * rstd
    h = np.abs(dy64 * w64).max(-1, keepdims=True)
    assert np.all(np.abs(np64(got[0]) - dx) <= 100 * U * rstd * h * (1 + z * z) + HALF[got[0].dtype] * np.abs(dx) * 1.01)
    tw = HALF[got[1].dtype]
    assert np.all(np.abs(np64(got[1]) - dw) <= 2e-6 * (np.abs(dy64) * z).sum(0) + tw * np.abs(dw) * 1.01)
    assert (got[2] is None) == (not bias)
    if bias:
        assert np.all(np.abs(np64(got[2]) - db) <= 2e-6 * np.abs(dy64).sum(0) + tw * np.abs(db) * 1.01)


SIZES = [(1, 1), (3, 7), (1, 8), (5, 64), (33, 129), (1000, 100), (7, 128), (9, 256), (4, 264), (17, 512), (65, 1000),
         (13, 1024), (21, 1500), (6, 2048), (3, 4097), (5, 4096), (2, 8192), (3, 8200), (2, 16384), (2, 16383)]


@pytest.mark.parametrize("t,wt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                  (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("rows,D", SIZES)
def test_sizes(rows, D, t, wt):
    x, w, b, dy = make(rows, D, t, wt, rows * 131 + D)
    for bias in (b, None):
        y = torch.full_like(x, float("nan"))
        api.infini_attn_layer_norm_forward(x, w, bias, y, eps=1e-5)
        check_forward(x, w, bias, y, 1e-5)
    check_backward(x, w, dy, api.infini_attn_layer_norm_backward(x, w, dy, eps=1e-5), 1e-5)
    check_backward(x, w, dy, api.infini_attn_layer_norm_backward(x, w, dy, eps=1e-5, want_bias=False), 1e-5, False)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(9001, 77), (5003, 1001), (2500, 2341), (1201, 8190), (20000, 12), (7, 16379), (5, 1), (4001, 3), (9, 5)])
def test_many_rows_that_start_anywhere(rows, D, t):
    x, w, b, dy = make(rows, D, t, t, rows)
    y = torch.full_like(x, float("nan"))
    api.infini_attn_layer_norm_forward(x, w, b, y)
    check_forward(x, w, b, y, 1e-5)
    check_backward(x, w, dy, api.infini_attn_layer_norm_backward(x, w, dy), 1e-5)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_tensors_on_different_grids(t):
    x, w, b, _ = make(50, 130, t, t, 5)
    for shift in (1, 3):
        y = torch.zeros(50 * 130 + 8, dtype=t, device=DEV)
        api.infini_attn_layer_norm_forward(x, w, b, y[shift:shift + 50 * 130].view(50, 130))
        check_forward(x, w, b, y[shift:shift + 50 * 130].view(50, 130), 1e-5)
        assert not y[:shift].any() and not y[shift + 50 * 130:].any()


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(11, 512), (13, 1), (6, 3), (40, 77)])
def test_pointers_off_alignment(rows, D, t):
    x, w, b, dy = make(rows, D, t, t, 3, shift=1)
    y = torch.empty(rows * D + 1, dtype=t, device=DEV)[1:].view(rows, D)
    api.infini_attn_layer_norm_forward(x, w, b, y)
    check_forward(x, w, b, y, 1e-5)
    check_backward(x, w, dy, api.infini_attn_layer_norm_backward(x, w, dy), 1e-5)


def test_large_mean_and_constant_rows():
    x, w, b, _ = make(8, 768, torch.float32, torch.float32, 9, mean=1000.0)
    x[3] = 7.25  # no spread at all: y is the bias
    y = torch.empty_like(x)
    api.infini_attn_layer_norm_forward(x, w, b, y)
    check_forward(x, w, b, y, 1e-5)
    assert torch.equal(y[3], b)


def test_many_rows_and_in_place():
    x, w, b, dy = make(70001, 72, torch.bfloat16, torch.float32, 4)
    got = api.infini_attn_layer_norm_backward(x, w, dy)
    check_backward(x, w, dy, got, 1e-5)
    again = api.infini_attn_layer_norm_backward(x, w, dy)
    assert all(torch.equal(a, c) for a, c in zip(got, again))
    y = torch.empty_like(x)
    api.infini_attn_layer_norm_forward(x, w, b, y)
    api.infini_attn_layer_norm_forward(x, w, b, x)
    assert torch.equal(x, y)


def test_a_bad_row_stays_in_its_row():
    x, w, b, dy = make(6, 320, torch.bfloat16, torch.bfloat16, 8)
    y0, y1 = torch.empty_like(x), torch.empty_like(x)
    api.infini_attn_layer_norm_forward(x, w, b, y0)
    x[2, 17] = float("inf")
    x[4, 0] = float("nan")
    api.infini_attn_layer_norm_forward(x, w, b, y1)
    good = [0, 1, 3, 5]
    assert torch.equal(y0[good], y1[good]) and torch.isnan(y1[4]).all() and torch.isnan(y1[2]).any()


def test_stream_workspace_and_graph():
    x, w, b, dy = make(300, 1024, torch.bfloat16, torch.float32, 21)
    want = api.infini_attn_layer_norm_backward(x, w, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = api.infini_attn_layer_norm_backward_workspace_size(300, 1024)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    got = api.infini_attn_layer_norm_backward(x, w, dy, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    y = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.infini_attn_layer_norm_forward(x, w, b, y)
        held = api.infini_attn_layer_norm_backward(x, w, dy, workspace=ws)
    x2, _, _, dy2 = make(300, 1024, torch.bfloat16, torch.float32, 22)
    x.copy_(x2)
    dy.copy_(dy2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check_forward(x, w, b, y, 1e-5)
    check_backward(x, w, dy, held, 1e-5)


def test_norm_in_front_of_the_layer():
    """The layer's pre-norm: a residual stream, normalised, through the projections and the memory, against the fp64
    oracle of the layer on the oracle's norm rounded to bf16.  The layer's own tolerances (max-abs 2e-2, relative L2
    5e-3) hold: an input that rounds the other way is one bf16 step off in one of D products."""
    from compressive_memory_transformer_sm_b200 import DELTA
    from compressive_memory_transformer_sm_b200 import workloads as W
    from oracle import infini_ref as R

    B, H, L, N, D = 1, 2, 384, 128, 256
    x, w_qkv, w_o, beta = (t.to(DEV) for t in W.make_layer_inputs(B, H, L, D, seed=9300))
    x = (3 * x + 1).contiguous()
    w, b = (1 + 0.2 * torch.randn(D, device=DEV)).bfloat16(), (0.1 * torch.randn(D, device=DEV)).bfloat16()
    y, out = torch.empty_like(x), torch.empty_like(x)
    M, z = torch.zeros(B, H, 128, 128, device=DEV), torch.zeros(B, H, 128, device=DEV)
    api.infini_attn_layer_norm_forward(x, w, b, y)
    api.infini_attn_layer_forward(y, w_qkv, w_o, beta, M, z, out, H, N, DELTA)
    torch.cuda.synchronize()
    norm = torch.from_numpy(G.layer_norm(np64(x), np64(w), np64(b), 1e-5)).bfloat16()
    wy, wM, _ = R.layer_forward(np64(norm), np64(w_qkv), np64(w_o), np64(beta), H, N, mode=DELTA, M0=np64(M) * 0, z0=np64(z) * 0)
    got = np64(out)
    assert np.abs(got - wy).max() <= 2e-2 * max(1.0, np.abs(wy).max())
    assert np.linalg.norm(got - wy) <= 5e-3 * np.linalg.norm(wy)
    assert np.linalg.norm(np64(M) - wM) <= 5e-3 * np.linalg.norm(wM)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,D", [(3, 64), (5, 100), (9, 256), (17, 512), (7, 1000), (1, 24)])
def test_eps_zero(rows, D, t):
    """Blocks hold several short rows at once: places without a row add nothing to the weights' gradients."""
    x, w, b, dy = make(rows, D, t, torch.float32, 7 * rows + D)
    y = torch.empty_like(x)
    api.infini_attn_layer_norm_forward(x, w, b, y, eps=0.0)
    check_forward(x, w, b, y, 0.0)
    check_backward(x, w, dy, api.infini_attn_layer_norm_backward(x, w, dy, eps=0.0), 0.0)
