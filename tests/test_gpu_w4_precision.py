"""moe_expert_ffn_w4: what its activations are rounded to, in every form (one token, a few rows, many rows)."""

import numpy as np
import pytest
import torch

from helpers import np64
from oracle import block_oracle as O
from test_gpu_w4 import B, DT, Layer, U, activations, check, routing  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k", [(1, 2), (1, 8), (4, 3), (20, 2)])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("kind", ["bf16", "q8", "f32"])
@pytest.mark.parametrize("large", ["x", "a"])
def test_neighbours_of_a_large_value_keep_their_bits(B, large, kind, group, T, k):  # noqa: F811
    """One input of the experts (or of their second product, `a`) is some 2000 times the others, and its weights are zero: each
    output holds what the others add."""
    h, f = 256, 96
    layer = Layer(B, 8, h, f, group, DT[kind])
    for i in (0, 1) if large == "x" else (2,):
        q, s = layer.mats[i]
        q[:, :, 4] = (q[:, :, 4] & 0xF0) | 8  # the nibble of input 8
    if large == "a":
        for i in (0, 1):
            layer.mats[i][1][:, 8] *= 45
    layer.dense = [O.weights_w4(q.cpu().numpy(), s.float().cpu().numpy(), group) for q, s in layer.mats]
    if kind == "q8":
        x = (torch.randn(T, h, generator=torch.Generator("cuda").manual_seed(5), device="cuda") * 0.2).to(torch.float8_e4m3fn)
        xs = torch.full((T, h // 128), 4.0, device="cuda")
        if large == "x":
            x[:, 8] = 448.0
        X = x.float().cpu().numpy().astype(np.float64) * 4.0
    else:
        x, xs, _ = activations(T, h, kind, 5)
        if large == "x":
            x[:, 8] = 2000.0
        X = np64(x)
    idx, w = routing(T, 8, k, 5)
    y = np64(layer.run(B, x, xs, idx, w, DT[kind]))
    want, A, Bd = O.expert_ffn_w4(X, idx.cpu().numpy(), np64(w), *layer.dense)
    # x: at most 2^-23 of itself, and 2^-24 of the largest of its 16 (a unit of 8355000 is 0.4% wider)
    ex = 1.01 * U * np.repeat(np.abs(X).reshape(T, h // 16, 16).max(2), 16, 1)
    W1, W3, W2 = layer.dense
    moved, most = np.zeros_like(y), np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e, c = int(idx[t, j]), float(w[t, j])
            z1, z3 = W1[e] @ X[t], W3[e] @ X[t]
            sig = 1.0 / (1.0 + np.exp(-z1))
            moved[t] += c * (np.abs(W2[e]) @ (1.1 * np.abs(z3) * (np.abs(W1[e]) @ ex[t]) + np.abs(z1 * sig) * (np.abs(W3[e]) @ ex[t])))
            a16 = np.repeat(np.abs(z1 * sig * z3).reshape(f // 16, 16).max(1), 16)
            most[t] += c * (np.abs(W2[e]) @ a16)
    # sums as in the tests of sizes; a: 11 bits in 16-bit layers, 23 in fp32 ones, and 2^-24 of the largest of its 16
    chain = lambda K: (24 + K / 1024 + 20) * 4 * U  # noqa: E731
    a_bits = 2.0 ** -11 if kind != "f32" else 2.0 ** -23
    half = torch.finfo(DT[kind]).eps / 2
    tol = chain(h) * Bd + (chain(f) + a_bits + (k + 8) * U) * A + 1.01 * U * most + moved
    assert (np.abs(y - want) <= tol + half * (np.abs(want) + tol)).all()


@pytest.mark.parametrize("T,k", [(1, 1), (1, 2), (4, 2), (20, 2)])
def test_every_output_of_one_weight_has_fp32_s_bits(B, T, k):  # noqa: F811
    """One weight for each output, of one: nothing is summed, and what is left of fp32 is what x and `a` were rounded to."""
    h = f = 64
    layer = Layer(B, 2, h, f, 32, torch.float32)
    at = np.arange(64)
    for i, source in enumerate((at, (at + 5) % 64, (at * 3 + 1) % 64)):
        q, s = layer.mats[i]
        codes = np.full((2, 64, 64), 8, np.uint8)
        codes[:, at, source] = 9
        q.copy_(torch.from_numpy(codes[:, :, 0::2] | (codes[:, :, 1::2] << 4)))
        s.fill_(1.0)
        layer.dense[i] = O.weights_w4(q.cpu().numpy(), s.float().cpu().numpy(), 32)
    # silu is the identity here; neighbours are within a factor of two of one another
    x = 32 + 32 * torch.rand(T, h, generator=torch.Generator("cuda").manual_seed(9), device="cuda")
    idx = torch.stack([torch.arange(k, dtype=torch.int32, device="cuda")] * T)
    w = torch.ones(T, k, device="cuda")
    y = np64(layer.run(B, x, None, idx, w, torch.float32))
    want, _, _ = O.expert_ffn_w4(np64(x), idx.cpu().numpy(), np64(w), *layer.dense)
    # two values of x: 2^-24 of twice their size, and 3 roundings each; a: 2^-24 of four times its size, 2 products, 3 roundings;
    # the sum over k
    assert (np.abs(y - want) <= (2 * (2 + 3) + (4 + 2 + 3) + 2) * U * np.abs(want)).all()


@pytest.mark.parametrize("k,h,f", [(8, 64, 4096), (8, 96, 7232), (3, 32, 20512), (64, 64, 960), (64, 64, 992), (1, 61440, 32), (2, 64000, 32)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_one_token_at_the_edge_of_shared_memory(B, kind, k, h, f):  # noqa: F811
    check(B, Layer(B, k, h, f, 128, DT[kind]), 1, k, kind, seed=4)
