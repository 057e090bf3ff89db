"""moe_add_rmsnorm where a value of a row, or its scale, is at the edge of fp32."""

import numpy as np
import pytest
import torch

from helpers import np64
from oracle import block_oracle as O
from test_gpu_norm import DT, SUM, U, B, forward, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_tiny_products_of_rows_and_gamma(B, dt):  # noqa: F811
    """Rows of 1e-12 and gamma of 1e-28: s * gamma is below fp32's normal numbers, y and its scales are not."""
    T, h = 5, 328
    x = (rows(T, h, torch.float32, 1) * 1e-12).to(DT[dt])
    gamma = (1 + 0.2 * torch.randn(h, device="cuda", generator=torch.Generator("cuda").manual_seed(2))) * 1e-28
    x[:, 5] = 0
    _, y, q, qs, rstd = forward(B, x, None, gamma, eps=0.0, q8=True)
    v, rs = O.rmsnorm(np64(x), np64(gamma), 0.0)
    # as in the tests of ordinary rows: mean of squares, root, division and products
    rel = (SUM / 2 + 4) * U
    half = torch.finfo(x.dtype).eps / 2
    assert (np.abs(np64(rstd) - rs) <= rel * rs).all()
    assert (np.abs(np64(y) - v) <= (half * (1 + 1e-3) + rel + 3 * U) * np.abs(v)).all()
    scale = O.q8_scales(v)
    assert (np.abs(np64(qs) - scale) <= (rel + 4 * U) * scale).all()
    got = q.float().cpu().numpy().astype(np.float64) * np.repeat(np64(qs), 128, 1)[:, :h]
    tol = (2.0 ** -4 + 2 * rel + 8 * U) * np.abs(v) + 2.0 ** -10 * np.repeat(scale, 128, 1)[:, :h]
    assert (np.abs(got - v) <= tol).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scales_beside_nan(B, dt):  # noqa: F811
    """A NaN of the row is in its rstd, and so in all of y and q: its scales are the smallest there is.  One of gamma stays in
    its column, and its group's scale is that of the other columns."""
    T, h = 3, 384
    x, gamma = rows(T, h, DT[dt], 1), torch.ones(h, device="cuda")
    clean = forward(B, x, None, gamma, q8=True)
    bad = x.clone()
    bad[1, 200] = float("nan")
    _, y, q, qs, rstd = forward(B, bad, None, gamma, q8=True)
    assert torch.isnan(y[1]).all() and torch.isnan(q[1].float()).all() and torch.isnan(rstd[1])
    assert (qs[1] == 2.0 ** -100 / 448).all()
    for t in (0, 2):
        assert torch.equal(y[t], clean[1][t]) and torch.equal(qs[t], clean[3][t])
    where = int(x[0, 128:256].abs().argmin()) + 128
    gamma[where] = float("nan")
    _, y, q, qs, _ = forward(B, x, None, gamma, q8=True)
    for out in (y.float(), q.float()):
        assert torch.isnan(out[:, where]).all() and int(torch.isnan(out).sum()) == T
    assert torch.equal(qs[0], clean[3][0])
