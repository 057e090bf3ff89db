"""moe_expert_ffn_w4 with many rows: the same call gives the same bits, and a row's sums go by the routing alone."""

import pytest
import torch

from test_gpu_w4 import B, DT, Layer, activations, routing  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "q8", "f32"])
def test_the_same_call_gives_the_same_bits(B, group, kind):  # noqa: F811
    # 200 rows of 2, most of them of a few experts: full units of rows, and shorter ones behind them
    layer = Layer(B, 16, 512, 512, group, DT[kind])
    x, xs, _ = activations(200, 512, kind, 3)
    idx, w = routing(200, 16, 2, 3, 1.0)
    want = layer.run(B, x, xs, idx, w, DT[kind])
    for _ in range(30):
        assert torch.equal(layer.run(B, x, xs, idx, w, DT[kind]).view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("group", [64, 128])
def test_an_expert_s_last_rows_are_its_short_unit(B, group):  # noqa: F811
    """Weights of one and three inputs whose sum shows its order: 2^17, and in the next eight inputs its negative and a small
    number.  One sum over all of them ends at the small number, a sum of every other eight inputs does not hold it beside 2^17.
    What the first 192 of an expert's 200 rows get is what 192 rows get."""
    T, h, f = 200, 128, 128
    layer = Layer(B, 2, h, f, group, torch.bfloat16)
    for q, s in layer.mats[:2]:
        q.fill_(0x99)
        s.fill_(1.0)
    x = torch.zeros(T, h, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 8] = 2.0 ** 17, -2.0 ** 17
    x[:, 10] = 2.0 ** -10 * (1 + torch.arange(T, device="cuda") % 7)
    idx = torch.ones(T, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(T, 1, device="cuda")
    want = layer.run(B, x[:192].contiguous(), None, idx[:192], w[:192], torch.bfloat16)
    for _ in range(30):
        assert torch.equal(layer.run(B, x, None, idx, w, torch.bfloat16)[:192], want)
