"""moe_add_rmsnorm and its backward on the GPU against the fp64 oracle.

Tolerances count roundings of 2^-24 (fp32) and eps/2 of the output's type.  A row's sum of h terms is taken in chains of
at most 32 in a thread, 5 in a warp and 32 over warps: 70 roundings bound it."""

import numpy as np
import pytest
import torch

from helpers import np64
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SUM = 70
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_pft_gb300 import binding, build

    build.build()
    return binding


def rows(T, h, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, h, generator=g, device="cuda") * std
    x[:, ::37] *= 10
    return x.to(dtype)


def forward(B, x, r, gamma, eps=1e-6, q8=False, y=True, in_place=False):
    T, h = x.shape
    nan = float("nan")
    s = None if r is None else (r if in_place else torch.full_like(x, nan))
    y = torch.full_like(x, nan) if y else None
    q = torch.zeros(T, h, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) if q8 else None
    qs = torch.full((T, -(-h // 128)), nan, device="cuda") if q8 else None
    rstd = torch.full((T,), nan, device="cuda")
    ws = B.new_workspace(B.MOE_OP_ADD_RMSNORM, T, h, 1, 1, 0, x.dtype)
    B.moe_add_rmsnorm(x, r, gamma, eps, s, y, q, qs, rstd, ws)
    return s, y, q, qs, rstd


SHAPES = [(1, 8), (1, 7168), (3, 64), (5, 1000), (2, 1032), (7, 16384), (33, 128), (300, 136), (257, 2048), (1, 4104), (6, 8192)]


@pytest.mark.parametrize("T,h", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res,q8", [(True, True), (False, False), (True, False), (False, True)])
def test_forward(B, T, h, dt, res, q8):
    x, gamma = rows(T, h, DT[dt], 1), 1 + 0.2 * torch.randn(h, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    r = rows(T, h, DT[dt], 3, 2.0) if res else None
    want_s = (x.float() + r.float()).to(x.dtype) if res else x
    s, y, q, qs, rstd = forward(B, x, r, gamma, q8=q8)
    if res:
        assert torch.equal(s, want_s)
    v, rs = O.rmsnorm(np64(want_s), np64(gamma), 1e-6)
    # mean of squares: SUM + 2 roundings, halved by the root; root, division and product
    rel = (SUM / 2 + 4) * U
    assert (np.abs(np64(rstd) - rs) <= rel * rs).all()
    half = torch.finfo(x.dtype).eps / 2
    assert (np.abs(np64(y) - v) <= (half * (1 + 1e-3) + rel + 3 * U) * np.abs(v)).all()
    if q8:
        scale = O.q8_scales(v)
        assert (np.abs(np64(qs) - scale) <= (rel + 4 * U) * scale).all()
        got = q.float().cpu().numpy().astype(np.float64) * np.repeat(np64(qs), 128, 1)[:, :h]
        # e4m3: half a step of 2^-4 relative, or of the subnormal grid 2^-9
        tol = (2.0 ** -4 + 2 * rel + 8 * U) * np.abs(v) + 2.0 ** -10 * np.repeat(scale, 128, 1)[:, :h]
        assert (np.abs(got - v) <= tol).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_forward_in_place_and_eight_bits_alone(B, in_place):
    x, r, gamma = rows(9, 512, torch.bfloat16, 5), rows(9, 512, torch.bfloat16, 6), torch.ones(512, device="cuda")
    want = (x.float() + r.float()).to(x.dtype)
    full = forward(B, x, r.clone(), gamma, q8=True)
    s, y, q, qs, _ = forward(B, x, r, gamma, q8=True, y=False, in_place=in_place)
    assert y is None and torch.equal(s, want)
    assert torch.equal(q.view(torch.uint8), full[2].view(torch.uint8)) and torch.equal(qs, full[3])


def test_forward_rows_of_zeros_infinities_and_nan(B):
    x = rows(6, 256, torch.bfloat16, 7)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    x[3] = torch.finfo(torch.bfloat16).max  # its square overflows: the row's rstd is 0
    gamma = torch.ones(256, device="cuda")
    _, y, q, qs, rstd = forward(B, x, None, gamma, q8=True)
    clean = forward(B, x[4:].contiguous(), None, gamma, q8=True)
    assert torch.equal(y[4:], clean[1]) and torch.equal(qs[4:], clean[3])  # rows do not see one another
    assert (y[0] == 0).all() and (q[0].float() == 0).all() and torch.isfinite(qs[0]).all()
    assert torch.isnan(y[1]).all() and torch.isnan(q[1].float()).all()
    assert rstd[2] == 0 and torch.isnan(y[2, 200]) and (y[2, :200] == 0).all()
    assert (y[3] == 0).all()


def test_empty_batch(B):
    x = torch.zeros(0, 64, device="cuda")
    forward(B, x, None, torch.ones(64, device="cuda"))
    dgamma = torch.full((64,), 3.0, device="cuda")
    ws = B.new_workspace(B.MOE_OP_ADD_RMSNORM_BWD, 0, 64, 1, 1, 0, torch.float32)
    B.moe_add_rmsnorm_bwd(x, x, torch.ones(64, device="cuda"), torch.zeros(0, device="cuda"), None, x.clone(), dgamma, ws)
    assert (dgamma == 0).all()


def backward(B, dy, s, gamma, rstd, add, in_place=False):
    T, h = s.shape
    ds = add if in_place else torch.full_like(s, float("nan"))
    dgamma = torch.full((h,), float("nan"), device="cuda")
    ws = B.new_workspace(B.MOE_OP_ADD_RMSNORM_BWD, T, h, 1, 1, 0, s.dtype)
    ws[256:] = 255  # what an earlier call left there
    B.moe_add_rmsnorm_bwd(dy, s, gamma, rstd, add, ds, dgamma, ws)
    return ds, dgamma


@pytest.mark.parametrize("T,h", SHAPES + [(1533, 1000), (4099, 72), (700, 7168)])
@pytest.mark.parametrize("dt,add", [("bf16", True), ("bf16", False), ("f32", True), ("f32", False)])
def test_backward(B, T, h, dt, add):
    s, dy = rows(T, h, DT[dt], 11), rows(T, h, DT[dt], 12)
    a = rows(T, h, DT[dt], 13) if add else None
    gamma = 1 + 0.2 * torch.randn(h, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    rstd = (s.double().square().mean(1) + 1e-6).rsqrt().float()
    ds, dgamma = backward(B, dy, s, gamma, rstd, a)
    S, D, G, R = np64(s), np64(dy), np64(gamma), np64(rstd)
    want, want_g = O.rmsnorm_bwd(D, S, G, R, np64(a) if add else None)
    xh, g = S * R[:, None], D * G
    terms = np.abs(R[:, None] * g) + np.abs(R[:, None] * xh) * np.abs((g * xh).mean(1, keepdims=True)) + (np.abs(np64(a)) if add else 0)
    mean_err = (SUM + 4) * U * np.abs(g * xh).mean(1, keepdims=True)
    half = torch.finfo(s.dtype).eps / 2
    tol = half * np.abs(want) * (1 + 1e-3) + 8 * U * terms + np.abs(R[:, None] * xh) * mean_err
    assert (np.abs(np64(ds) - want) <= tol + half * tol).all()
    # dgamma: at most T + 64 additions in a chain, and 2 roundings a term
    assert (np.abs(np64(dgamma) - want_g) <= (T + 66) * U * np.abs(D * xh).sum(0)).all()
    again = backward(B, dy, s, gamma, rstd, a)
    assert torch.equal(ds, again[0]) and torch.equal(dgamma, again[1])
    if add:
        assert torch.equal(backward(B, dy, s, gamma, rstd, a.clone(), in_place=True)[0], ds)


def test_backward_is_the_forward_s_derivative(B):
    T, h = 4, 96
    x, gamma, dy = rows(T, h, torch.float32, 21), torch.rand(h, device="cuda") + 0.5, rows(T, h, torch.float32, 22)
    _, _, _, _, rstd = forward(B, x, None, gamma, eps=1e-5)
    ds, dgamma = backward(B, dy, x, gamma, rstd, None)
    r = np.random.RandomState(3)
    X, G, D = np64(x), np64(gamma), np64(dy)
    f = lambda X, G: float((O.rmsnorm(X, G, 1e-5)[0] * D).sum())  # noqa: E731
    for _ in range(4):
        u, w, d = r.randn(T, h), r.randn(h), 1e-5
        num = (f(X + d * u, G + d * w) - f(X - d * u, G - d * w)) / (2 * d)
        got = (np64(ds) * u).sum() + (np64(dgamma) * w).sum()
        # fp32 gradients: 100 roundings of the sum of absolute terms
        assert abs(num - got) <= 100 * U * (np.abs(np64(ds) * u).sum() + np.abs(np64(dgamma) * w).sum()) + 1e-6 * abs(num) + 1e-6


def test_captured_and_on_another_stream(B):
    x, r, gamma = rows(40, 1024, torch.bfloat16, 31), rows(40, 1024, torch.bfloat16, 32), torch.ones(1024, device="cuda")
    s, y, _, _, rstd = forward(B, x, r, gamma)
    ds, dg = backward(B, y, s, gamma, rstd, r)
    y2, s2, rs2, ds2, dg2 = (torch.zeros_like(t) for t in (y, s, rstd, ds, dg))
    ws = B.new_workspace(B.MOE_OP_ADD_RMSNORM_BWD, 40, 1024, 1, 1, 0, x.dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        B.moe_add_rmsnorm(x, r, gamma, 1e-6, s2, y2, None, None, rs2, ws)
        B.moe_add_rmsnorm_bwd(y2, s2, gamma, rs2, r, ds2, dg2, ws)

    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(ds2, ds) and torch.equal(dg2, dg)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for t in (y2, s2, rs2, ds2, dg2):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ds2, ds) and torch.equal(dg2, dg) and torch.equal(y2, y)
