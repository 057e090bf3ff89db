"""The operators around the MoE layer on the CPU: add + RMSNorm and its adjoint, the AdamW step with 32- and 8-bit
states, and the routed experts over 4-bit weights.

NumPy in fp64, from the formulas of include/moe_pft.h.  What the library defines bit by bit (the 8-bit states, whose
codes come from single fp32 operations and Philox words) is restated in fp32 operations of NumPy, each correctly rounded.
"""

from __future__ import annotations

import numpy as np

# ------------------------------------------------------------------------------------------ norm


def rmsnorm(s, gamma, eps):
    """(v, rstd) of rows s: v = s * rstd * gamma."""
    rstd = 1.0 / np.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * gamma, rstd


def rmsnorm_bwd(dy, s, gamma, rstd, ds_add=None):
    xh, g = s * rstd[:, None], dy * gamma
    ds = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdims=True))
    return (ds if ds_add is None else ds + ds_add), (dy * xh).sum(0)


def q8_scales(v, group=128):
    n = -(-v.shape[1] // group)
    p = np.pad(np.abs(v), ((0, 0), (0, n * group - v.shape[1]))).reshape(v.shape[0], n, group)
    return np.maximum(p.max(2), 2.0 ** -100) / 448.0


# ------------------------------------------------------------------------------------------ AdamW


def philox7(counter, seed):
    """Philox4x32 with 7 rounds; counter [n, 4] uint32, seed a 64-bit key; [n, 4] uint32."""
    c = counter.astype(np.uint64).T.copy()
    k = [np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32 & 0xFFFFFFFF)]
    mask, m0, m1 = np.uint64(0xFFFFFFFF), np.uint64(0xD2511F53), np.uint64(0xCD9E8D57)
    s = np.uint64(32)
    for _ in range(7):
        a, b = c[0] * m0, c[2] * m1
        c = np.stack([(b >> s) ^ c[1] ^ k[0], b & mask, (a >> s) ^ c[3] ^ k[1], a & mask])
        k = [(k[0] + np.uint64(0x9E3779B9)) & mask, (k[1] + np.uint64(0xBB67AE85)) & mask]
    return c.T.astype(np.uint32)


def random_words(n, tensor, step, seed):
    """The 32 random bits of each of a tensor's n elements."""
    q = np.arange(-(-n // 4), dtype=np.uint64)
    c = np.stack([q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), np.full_like(q, tensor), np.full_like(q, step)], 1)
    return philox7(c.astype(np.uint32), seed).reshape(-1)[:n]


def adamw(p, g, m, v, lr, step, wd, b1, b2, eps, grad_scale=1.0):
    """(p, m, v) after the step, fp64."""
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    u = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p - lr * (wd * p + u), m, v


def _f32(x):
    return np.float32(x)


def adamw_states_f32(g, m, v, b1, b2, grad_scale=1.0):
    """m and v after the step in the library's fp32 operations."""
    g = _f32(g) * _f32(grad_scale)
    with np.errstate(over="ignore", invalid="ignore"):
        gg = g * g
    m1 = _f32(m) * _f32(b1) + g * _f32(1 - b1)
    v1 = _f32(v) * _f32(b2) + gg * _f32(1 - b2)
    ok = np.isfinite(gg)
    return np.where(ok, m1, _f32(m)), np.where(ok, v1, _f32(v))


def _blocks(x, block=256):
    n = -(-x.size // block)
    return np.pad(x, (0, n * block - x.size)).reshape(n, block)


def _round_random(x, bits16, drop, low):
    """x >= 0 (fp32) on 23 - drop mantissa bits, below `low` on the grid of [low, 2 low): random up or down."""
    small = x < _f32(low)
    b = np.where(small, x + _f32(low), x).view(np.uint32).astype(np.uint64)
    b = b + ((bits16.astype(np.uint64) << np.uint64(drop - 16)) | np.uint64(1 << (drop - 17)))
    r = (b & np.uint64(0xFFFFFFFF - ((1 << drop) - 1))).astype(np.uint32).view(np.float32)
    return np.where(small, r - _f32(low), r).astype(np.float32)


def quantize_states(m, v, words):
    """(codes of m, scale of m, codes of v, scale of v): the codes as the fp32 values of e4m3 and e5m2."""
    m, v = np.asarray(m, np.float32), np.asarray(v, np.float32)
    ms = np.maximum(np.abs(_blocks(m)).max(1), _f32(2.0 ** -100)) * _f32(2.0 ** -8)
    vs = np.maximum(_blocks(v).max(1), _f32(2.0 ** -100)) * _f32(2.0 ** -15)
    of = np.arange(m.size) // 256
    rm, rv = (_f32(1) / ms)[of], (_f32(1) / vs)[of]
    cm = np.copysign(_round_random(np.abs(m) * rm, words & np.uint32(0xFFFF), 20, 2.0 ** -6), m)
    cv = _round_random(v * rv, words >> np.uint32(16), 21, 2.0 ** -14)
    cv = np.where((v > 0) & (cv == 0), _f32(2.0 ** -16), cv)
    return cm, ms, cv, vs


# ------------------------------------------------------------------------------------------ 4-bit experts


def quantize_w4(W, group):
    """W [E, K, N] -> (q [E, N, K/2] uint8, scale [E, N, ceil(K/group)] fp32 holding bf16 values)."""
    import torch

    E, K, N = W.shape
    n = -(-K // group)
    w = np.pad(np.asarray(W, np.float32).transpose(0, 2, 1), ((0, 0), (0, 0), (0, n * group - K))).reshape(E, N, n, group)
    s = np.abs(w).max(3) / _f32(7.0)
    s = torch.from_numpy(s).to(torch.bfloat16).float().numpy()
    c = np.clip(np.rint(w / np.where(s == 0, _f32(1), s)[..., None]), -8, 7).astype(np.int32) + 8
    c = c.reshape(E, N, n * group)[:, :, :K].astype(np.uint8)
    return c[:, :, 0::2] | (c[:, :, 1::2] << 4), s


def weights_w4(q, scale, group):
    """[E, N, K] fp64."""
    c = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1).astype(np.float64) - 8.0
    return c * np.repeat(scale.astype(np.float64), group, -1)[..., :c.shape[-1]]


def expert_ffn_w4(x, topk_idx, topk_w, W1, W3, W2):
    """y and a bound on what fp32 sums and one rounding of `a` can move it by: (y, |terms| of the products).

    W1, W3 [E, f, h], W2 [E, h, f] fp64.  Returns y, and for each token the sums of absolute values that the error
    bounds scale with: (A, B), A = sum_j |w| |W2| |a|, B = sum_j |w| |W2| (|z3| (|W1||x|) + |silu(z1)| (|W3||x|))."""
    T, k = topk_idx.shape
    y = np.zeros((T, W2.shape[1]))
    A, Bd = np.zeros_like(y), np.zeros_like(y)
    for t in range(T):
        for j in range(k):
            e, w = topk_idx[t, j], float(topk_w[t, j])
            if not 0 <= e < W1.shape[0]:
                continue
            z1, z3 = W1[e] @ x[t], W3[e] @ x[t]
            sig = 1.0 / (1.0 + np.exp(-z1))
            a = z1 * sig * z3
            y[t] += w * (W2[e] @ a)
            W2a, ax = np.abs(W2[e]), np.abs(x[t])
            A[t] += abs(w) * (W2a @ np.abs(a))
            Bd[t] += abs(w) * (W2a @ (1.1 * np.abs(z3) * (np.abs(W1[e]) @ ax) + np.abs(z1 * sig) * (np.abs(W3[e]) @ ax)))
    return y, A, Bd
