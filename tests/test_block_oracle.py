"""The oracle of the operators around the layer against itself, on the CPU: gradients against differences, and the
properties that the 8-bit states are chosen for."""

import numpy as np

from oracle import block_oracle as O


def test_rmsnorm_gradient_against_differences():
    r = np.random.RandomState(1)
    T, h, eps = 5, 24, 1e-5
    x, gamma, dy, add = r.randn(T, h), 1 + 0.2 * r.randn(h), r.randn(T, h), r.randn(T, h)
    f = lambda x, gamma: float((O.rmsnorm(x, gamma, eps)[0] * dy).sum() + (x * add).sum())  # noqa: E731
    ds, dgamma = O.rmsnorm_bwd(dy, x, gamma, O.rmsnorm(x, gamma, eps)[1], add)
    d = 1e-5
    for _ in range(6):
        u, g = r.randn(T, h), r.randn(h)
        num = (f(x + d * u, gamma + d * g) - f(x - d * u, gamma - d * g)) / (2 * d)
        # central differences: third-order term ~ d^2, cancellation ~ 2^-52 |f| / d
        assert abs(num - (ds * u).sum() - (dgamma * g).sum()) <= 1e-6 * (abs(num) + 1)


def test_random_rounding_is_unbiased_and_keeps_v_positive():
    # a moving average whose steps are far below half a code: rounding to nearest would never move it
    v = np.full(256, 0.7, np.float32)
    v[0] = 1.0
    total = np.zeros(256)
    n = 400
    for step in range(1, n + 1):
        _, _, cv, vs = O.quantize_states(np.zeros(256, np.float32), v, O.random_words(256, 0, step, 99))
        total += cv * np.float64(vs[0])
    # one rounding is off by less than a code (a quarter of the binade's base, 0.5): sd of the mean of n * 255 <= 0.0625 / sqrt
    assert abs(total[1:].mean() / n - 0.7) <= 6 * 0.0625 / np.sqrt(255 * n)
    tiny = np.array([1.0] + [1e-30] * 255, np.float32)
    _, _, cv, _ = O.quantize_states(tiny, tiny, O.random_words(256, 0, 1, 3))
    assert (cv > 0).all()
    zero = np.zeros(256, np.float32)
    cm, _, cv, _ = O.quantize_states(zero, zero, O.random_words(256, 0, 1, 3))
    assert not cm.any() and not cv.any()


def test_codes_are_values_of_their_types():
    import torch

    r = np.random.RandomState(2)
    m = (r.randn(4096) * np.exp(4 * r.randn(4096))).astype(np.float32)
    cm, _, cv, _ = O.quantize_states(m, m * m, O.random_words(4096, 3, 17, 2 ** 40 + 5))
    for c, t in ((cm, torch.float8_e4m3fn), (cv, torch.float8_e5m2)):
        assert np.array_equal(torch.from_numpy(c).to(t).float().numpy(), c)


def test_quantized_weights_are_within_half_a_step():
    r = np.random.RandomState(4)
    W = r.randn(3, 96, 32).astype(np.float32)
    for group in (32, 64, 128):
        q, s = O.quantize_w4(W, group)
        got = O.weights_w4(q, s, group).transpose(0, 2, 1)
        step = np.repeat(s, group, 2)[:, :, :96].transpose(0, 2, 1)
        # half a step, and the largest value's cut where its scale was rounded down (bf16: 2^-9 of 7 steps)
        assert (np.abs(got - W) <= step * (0.5 + 7 * 2.0 ** -8)).all()
