"""moe_quantize_w4 at the small end of its scales."""

import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from test_gpu_w4 import B  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-29, 1e-31, 1e-34])
def test_tiny_weights(B, dtype, size):  # noqa: F811
    """Weights whose scale is far below any other number of a model are codes of that scale; a group of zeros has scale zero."""
    E, K, N, group = 2, 96, 64, 64
    W = (torch.randn(E, K, N, generator=torch.Generator("cuda").manual_seed(1), device="cuda") * size).to(dtype)
    W[1, :64, 7] = 0
    q = torch.full((E, N, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    s = torch.full((E, N, 2), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.moe_quantize_w4(W, group, q, s, torch.zeros(256, dtype=torch.uint8, device="cuda"))
    want_q, want_s = O.quantize_w4(W.float().cpu().numpy(), group)
    np.testing.assert_array_equal(s.float().cpu().numpy(), want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)
    assert want_s[1, 7, 0] == 0
    got = O.weights_w4(q.cpu().numpy(), want_s, group).transpose(0, 2, 1)
    step = np.repeat(want_s, group, 2)[:, :, :K].transpose(0, 2, 1)
    # half a step, and the largest value's cut where its scale was rounded down (bf16: 2^-8 of 7 steps)
    assert (np.abs(got - W.double().cpu().numpy()) <= step * (0.5 + 7 * 2.0 ** -8)).all()
