"""The block around the layer (block.py) on the GPU: its step against the oracles of its parts, its optimizer and its decode
step, and the example that runs them together."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from helpers import TOL, np64, rel_l2
from oracle import block_oracle as BO
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("block_example", os.path.join(ROOT, "examples", "block_train_and_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.build.build()
    return m


def test_forward_and_backward_against_the_oracles(example):
    from mixture_experts_layer_pft_gb300 import binding as B
    from mixture_experts_layer_pft_gb300 import block

    T, h, f, E, k = 96, 128, 64, 8, 2
    p = example.make_params(h, f, E, torch.float32, seed=3)
    b = block.BlockBuffers(T, h, E, k, f, torch.float32)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r, dy, ds = (torch.randn(T, h, generator=g, device="cuda") for _ in range(4))
    y, s = block.block_forward(p, x, r, b)
    dx = block.block_backward(p, dy, ds, b)
    assert B.moe_check_status(b.layer.ws) == 0 and B.moe_check_status(b.ws) == 0
    S = np64(x + r)
    n, rstd = BO.rmsnorm(S, np64(p["gamma"]), b.eps)
    W = [np64(p[v]) for v in ("Wg", "W1", "W3", "W2")]
    fw = O.layer_forward(n, *W, k, None, "f32")
    bw = O.layer_backward(fw, n, *W, np64(dy), "f32")
    want, dgamma = BO.rmsnorm_bwd(bw["dx"], S, np64(p["gamma"]), rstd, np64(ds))
    for got, ref in ((s, S), (y, fw["y"]), (dx, want), (b.dgamma, dgamma), (b.layer.dW2, bw["dW2"])):
        assert rel_l2(np64(got), ref) <= TOL["f32"]


@pytest.mark.parametrize("bits", [32, 8])
def test_training_lowers_the_loss_and_bits_agree(example, bits):
    p = example.make_params(256, 128, 8, torch.bfloat16)
    losses, _, _ = example.train(p, 256, 2, 40, bits)
    assert losses[-1] < 0.7 * losses[0] and all(np.isfinite(losses))
    q = example.make_params(256, 128, 8, torch.bfloat16)
    full, _, _ = example.train(q, 256, 2, 40, 32)
    assert abs(losses[-1] - full[-1]) <= 0.1 * full[0]  # 8-bit states follow the 32-bit ones


def test_captured_training_step_equals_the_eager_one(example):
    from mixture_experts_layer_pft_gb300 import block, layer

    def make():
        p = example.make_params(128, 64, 4, torch.bfloat16)
        b = block.BlockBuffers(64, 128, 4, 2, 64, torch.bfloat16)
        o = block.AdamW(*block.parameters(p, b), lr=1e-3, bits=8, seed=5)
        return p, b, o

    g = torch.Generator(device="cuda").manual_seed(4)
    x, r, d = (torch.randn(64, 128, generator=g, device="cuda").bfloat16() for _ in range(3))

    def step(p, b, o):
        block.block_forward(p, x, r, b)
        block.block_backward(p, d, d, b)
        o.step()

    a, c = make(), make()
    cap = layer.CapturedStep(lambda: step(*a), warmup=1)
    cap.replay()
    cap.replay()
    for _ in range(3):
        step(*c)
    torch.cuda.synchronize()
    for u, v in zip(a[2].masters + a[2].m + a[2].v, c[2].masters + c[2].m + c[2].v):
        if u is not None:
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


@pytest.mark.parametrize("dtype,act8", [(torch.bfloat16, True), (torch.bfloat16, False), (torch.float32, False)])
@pytest.mark.parametrize("T", [1, 3, 20])
def test_decode_is_the_layer_over_its_quantised_weights(example, dtype, act8, T):
    from mixture_experts_layer_pft_gb300 import block

    h, f, E, k, group = 256, 96, 8, 2, 32
    p = example.make_params(h, f, E, dtype, seed=6)
    dec = block.DecodeBlock(p, T, k, group=group, act8=act8)
    g = torch.Generator(device="cuda").manual_seed(7)
    x, r = (torch.randn(T, h, generator=g, device="cuda").to(dtype) for _ in range(2))
    y, s = dec.step(x, r)
    n = dec.n
    if act8:
        n = dec.q.float() * dec.q_scale.repeat_interleave(128, 1)[:, :h]
    dense = [BO.weights_w4(dec.w4[i].cpu().numpy(), dec.w4[i + 1].float().cpu().numpy(), group) for i in (0, 2, 4)]
    want, _, _ = BO.expert_ffn_w4(np64(n), dec.topk_idx.cpu().numpy(), np64(dec.topk_w), *dense)
    assert rel_l2(np64(y), want) <= TOL["f32" if dtype == torch.float32 else "bf16"]
    # 4 bits of normal weights: rounding errors of about a tenth
    W = [np64(p[v]).transpose(0, 2, 1) for v in ("W1", "W3", "W2")]
    full, _, _ = BO.expert_ffn_w4(np64(dec.n), dec.topk_idx.cpu().numpy(), np64(dec.topk_w), *W)
    assert rel_l2(np64(y), full) <= 0.3


def test_example(example, capsys):
    losses, off = example.main(["--tokens", "128", "--hidden", "256", "--ffn", "128", "--experts", "8", "--steps", "30"])
    assert losses[-1] < losses[0] and off < 0.3
    assert "decoded" in capsys.readouterr().out
