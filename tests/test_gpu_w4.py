"""moe_quantize_w4 and moe_expert_ffn_w4 on the GPU against the fp64 oracle over the same 4-bit weights."""

import numpy as np
import pytest
import torch

from helpers import np64
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "q8": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_pft_gb300 import binding, build

    build.build()
    return binding


def quantized(B, E, K, N, group, dtype, seed):
    W = (torch.randn(E, K, N, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") / K ** 0.5).to(dtype)
    q = torch.full((E, N, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    s = torch.full((E, N, -(-K // group)), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.moe_quantize_w4(W, group, q, s, ws)
    return W, q, s


@pytest.mark.parametrize("E,K,N", [(1, 32, 32), (3, 96, 160), (2, 128, 64), (2, 352, 96), (5, 64, 256)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize(B, E, K, N, group, dtype):
    W, q, s = quantized(B, E, K, N, group, dtype, 1)
    want_q, want_s = O.quantize_w4(W.float().cpu().numpy(), group)
    np.testing.assert_array_equal(s.float().cpu().numpy(), want_s)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q)


def test_quantize_zeros_and_values_that_are_no_numbers(B):
    W = torch.randn(1, 64, 32, device="cuda")
    W[0, :32, 3] = 0
    W[0, 5, 4] = float("nan")
    q = torch.zeros(1, 32, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, 32, 2, dtype=torch.bfloat16, device="cuda")
    B.moe_quantize_w4(W, 32, q, s, torch.zeros(256, dtype=torch.uint8, device="cuda"))
    got = O.weights_w4(q.cpu().numpy(), s.float().cpu().numpy(), 32)
    assert (got[0, 3, :32] == 0).all() and got[0, 4, 5] == 0 and np.isfinite(got).all()


class Layer:
    def __init__(self, B, E, h, f, group, dtype, seed=0):
        self.E, self.h, self.f, self.group = E, h, f, group
        self.mats = [quantized(B, E, K, N, group, dtype, seed + i)[1:] for i, (K, N) in enumerate([(h, f), (h, f), (f, h)])]
        self.dense = [O.weights_w4(q.cpu().numpy(), s.float().cpu().numpy(), group) for q, s in self.mats]

    def run(self, B, x, xs, idx, w, dtype, status=0):
        (W1q, W1s), (W3q, W3s), (W2q, W2s) = self.mats
        T, k = idx.shape
        y = torch.full((T, self.h), float("nan"), dtype=dtype, device="cuda")
        ws = B.new_workspace(B.MOE_OP_EXPERT_FFN_W4, T, self.h, self.E, k, self.f, dtype)
        ws[256:] = 255
        B.moe_expert_ffn_w4(x, xs, idx, w, W1q, W1s, W3q, W3s, W2q, W2s, self.group, y, ws)
        assert B.moe_check_status(ws) == status
        return y


def activations(T, h, kind, seed):
    x = torch.randn(T, h, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    x[:, ::29] *= 6
    if kind != "q8":
        return x.to(DT[kind]), None, np64(x.to(DT[kind]))
    xs = torch.rand(T, -(-h // 128), device="cuda") * 0.02 + 0.001
    q = (x / xs.repeat_interleave(128, 1)[:, :h]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q, xs, q.float().cpu().numpy().astype(np.float64) * np.repeat(np64(xs), 128, 1)[:, :h]


def routing(T, E, k, seed, skew=0.0):
    r = np.random.RandomState(seed)
    l = r.standard_normal((T, E)) - skew * np.log(np.arange(E) + 1.0)
    idx = np.argsort(-l, 1)[:, :k].astype(np.int32)
    w = r.rand(T, k).astype(np.float32)
    return torch.from_numpy(idx.copy()).cuda(), torch.from_numpy(w).cuda()


def check(B, layer, T, k, kind, seed=3, skew=0.0, idx=None, status=0):
    x, xs, X = activations(T, layer.h, kind, seed)
    own, w = routing(T, layer.E, k, seed, skew)
    idx = own if idx is None else idx
    y = layer.run(B, x, xs, idx, w, DT[kind], status)
    want, A, Bd = O.expert_ffn_w4(X, idx.cpu().numpy(), np64(w), *layer.dense)
    # a product's sums: mma chains of at most 8 a group (3 planes in fp32), then a step per 1024 inputs, 8 warps, k experts;
    # the tensor core's additions are counted as 2^-22 each.  a is rounded to its type once, y once.
    chain = lambda K: (24 + K / 1024 + 20) * 4 * U  # noqa: E731
    half = torch.finfo(DT[kind]).eps / 2
    tol = chain(layer.h) * Bd + (chain(layer.f) + half + (k + 8) * U) * A
    assert (np.abs(np64(y) - want) <= tol + half * (np.abs(want) + tol)).all()
    return y


@pytest.mark.parametrize("h,f", [(32, 32), (64, 96), (128, 64), (160, 224), (1056, 352), (2048, 192)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "q8", "f32"])
def test_sizes(B, h, f, group, kind):
    layer = Layer(B, 6, h, f, group, DT[kind])
    check(B, layer, 1, 1, kind)
    check(B, layer, 5, 3, kind, seed=4)


@pytest.mark.parametrize("T,k,skew", [(1, 8, 0.0), (2, 4, 0.0), (3, 2, 0.0), (7, 8, 1.6), (8, 1, 9.0), (9, 1, 9.0), (17, 2, 3.0),
                                      (64, 6, 1.6), (200, 2, 4.0), (700, 1, 50.0)])
@pytest.mark.parametrize("kind", ["bf16", "q8", "f32"])
def test_tokens(B, T, k, skew, kind):
    check(B, Layer(B, 16, 256, 128, 128, DT[kind]), T, k, kind, seed=T, skew=skew)


@pytest.mark.parametrize("E,T,k", [(40, 13, 3), (39, 13, 3), (38, 13, 3), (1024, 2, 8), (1, 5, 1)])
def test_slots_by_row_and_by_expert(B, E, T, k):
    check(B, Layer(B, E, 64, 64, 64, torch.bfloat16), T, k, "bf16", seed=6)


def test_rows_do_not_see_one_another(B):
    layer = Layer(B, 4, 128, 96, 64, torch.bfloat16)
    x, _, _ = activations(6, 128, "bf16", 8)
    idx, w = routing(6, 4, 2, 8)
    clean = layer.run(B, x, None, idx, w, torch.bfloat16)
    bad = x.clone()
    bad[2] = float("nan")
    bad[4, 7] = float("inf")
    y = layer.run(B, bad, None, idx, w, torch.bfloat16)
    for t in (0, 1, 3, 5):
        assert torch.equal(y[t], clean[t])
    assert torch.isnan(y[2]).all()
    for t in range(6):  # nor does the batch change a row
        assert torch.equal(layer.run(B, x[t:t + 1].contiguous(), None, idx[t:t + 1].contiguous(), w[t:t + 1].contiguous(), torch.bfloat16)[0], clean[t])


@pytest.mark.parametrize("E", [4, 64])
def test_bad_and_repeated_experts(B, E):
    layer = Layer(B, E, 64, 64, 32, torch.bfloat16)
    idx = routing(5, E, 2, 9)[0]
    idx[1, 0], idx[2, 1], idx[3, 0], idx[3, 1] = -1, E, 2 ** 31 - 1, -2 ** 31
    y = check(B, layer, 5, 2, "bf16", idx=idx, status=B.MOE_STATUS_BAD_INDEX)
    assert (y[3] == 0).all()
    idx = torch.full((3, 2), 2, dtype=torch.int32, device="cuda")
    check(B, layer, 3, 2, "bf16", idx=idx)


def test_norm_s_eight_bits_feed_the_experts(B):
    layer = Layer(B, 8, 384, 128, 128, torch.bfloat16)
    x = torch.randn(3, 384, device="cuda").bfloat16()
    q, qs = torch.empty(3, 384, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(3, 3, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.moe_add_rmsnorm(x, None, torch.ones(384, device="cuda"), 1e-6, None, None, q, qs, None, ws)
    idx, w = routing(3, 8, 2, 1)
    y = layer.run(B, q, qs, idx, w, torch.bfloat16)
    want, _, _ = O.expert_ffn_w4(q.float().cpu().numpy().astype(np.float64) * np.repeat(np64(qs), 128, 1), idx.cpu().numpy(), np64(w), *layer.dense)
    assert np.linalg.norm(np64(y) - want) <= 2 ** -7 * np.linalg.norm(want)  # two bf16 roundings


def test_captured_and_repeatable(B):
    layer = Layer(B, 8, 256, 160, 64, torch.bfloat16)
    x, _, _ = activations(4, 256, "bf16", 8)
    idx, w = routing(4, 8, 2, 8)
    want = layer.run(B, x, None, idx, w, torch.bfloat16)
    (W1q, W1s), (W3q, W3s), (W2q, W2s) = layer.mats
    y = torch.zeros_like(want)
    ws = B.new_workspace(B.MOE_OP_EXPERT_FFN_W4, 4, 256, 8, 2, 160, torch.bfloat16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            B.moe_expert_ffn_w4(x, None, idx, w, W1q, W1s, W3q, W3s, W2q, W2s, 64, y, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    empty = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    layer.run(B, empty, None, idx[:0], w[:0], torch.bfloat16)


@pytest.mark.parametrize("h,f", [(32, 32), (64, 96), (160, 224), (1056, 352), (2048, 192)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "q8", "f32"])
def test_twelve_rows(B, h, f, group, kind):
    check(B, Layer(B, 6, h, f, group, DT[kind]), 4, 3, kind, seed=5)


@pytest.mark.parametrize("E,T,k,h,f", [(40, 60, 4, 128, 2048), (40, 60, 4, 2048, 128), (24, 40, 2, 320, 1056), (3, 64, 1, 96, 64)])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("kind", ["bf16", "q8", "f32"])
def test_many_and_few_items(B, E, T, k, h, f, group, kind):
    check(B, Layer(B, E, h, f, group, DT[kind]), T, k, kind, seed=7)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_many_rows_do_not_see_one_another(B, kind):
    layer = Layer(B, 4, 160, 96, 32, DT[kind])
    x, _, _ = activations(21, 160, kind, 8)
    idx, w = routing(21, 4, 2, 8)
    clean = layer.run(B, x, None, idx, w, DT[kind])
    bad = x.clone()
    bad[2] = float("nan")
    bad[4, 7] = float("inf")
    y = layer.run(B, bad, None, idx, w, DT[kind])
    keep = [t for t in range(21) if t not in (2, 4)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[2]).all()


def test_bad_experts_among_many_rows(B):
    layer = Layer(B, 8, 64, 64, 32, torch.bfloat16)
    idx = routing(30, 8, 2, 9)[0]
    idx[1, 0], idx[2, 1], idx[3, 0], idx[3, 1] = -1, 8, 2 ** 31 - 1, -2 ** 31
    y = check(B, layer, 30, 2, "bf16", idx=idx, status=B.MOE_STATUS_BAD_INDEX)
    assert (y[3] == 0).all()


@pytest.mark.parametrize("T,k", [(1, 2), (4, 3), (20, 2)])
def test_a_large_value_that_meets_zero_weights(B, T, k):
    """An input 2000 times the others whose weights are zero in every expert: what the others add is not lost beside it."""
    layer = Layer(B, 4, 128, 64, 128, torch.bfloat16)
    for i in (0, 1):
        q = layer.mats[i][0]
        q[:, :, 4] = (q[:, :, 4] & 0xF0) | 8  # the nibble of input 8
        layer.dense[i] = O.weights_w4(q.cpu().numpy(), layer.mats[i][1].float().cpu().numpy(), 128)
    x, _, _ = activations(T, 128, "bf16", 3)
    x[:, 8] = 2000.0
    idx, w = routing(T, 4, k, 3)
    y = layer.run(B, x, None, idx, w, torch.bfloat16)
    want, A, _ = O.expert_ffn_w4(np64(x), idx.cpu().numpy(), np64(w), *layer.dense)
    # x is off by at most 2^-16 of 2000 (0.03 beside values of 1) in 16 of 128 inputs, a by 2^-8, y by 2^-8: an eighth of the
    # row's largest output holds the sum of these for a dot product of 128 terms
    assert np.abs(np64(y) - want).max() <= np.abs(want).max() / 8
