"""moe_adamw_step on the GPU: fp64 formulas for what is rounded to fp32, and bit for bit for the 8-bit states."""

import numpy as np
import pytest
import torch

from helpers import np64
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
B1, B2, EPS = 0.9, 0.999, 1e-8


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_pft_gb300 import binding, build

    build.build()
    return binding


class Model:
    """Tensors of the given sizes and types with gradients and states, on the GPU."""

    def __init__(self, sizes, dtypes, bits, seed=0, fresh=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
        self.bits, self.sizes, self.dtypes = bits, sizes, dtypes
        self.masters, self.params, self.grads = [], [], []
        self.m, self.v = [], []
        self.ms, self.vs = ([], []) if bits == 8 else (None, None)
        for n, d in zip(sizes, dtypes):
            p, gr = rn(n) * 0.05, rn(n) * torch.exp(rn(n))
            self.grads.append(gr.to(d))
            self.masters.append(p if d == torch.bfloat16 else None)
            self.params.append(p.to(d) if d == torch.bfloat16 else p)
            m, v = rn(n) * 0.1, rn(n).square() * 0.3
            if fresh:
                m, v = m * 0, v * 0
            if bits == 8:
                nb = -(-n // 256)
                of = torch.arange(n, device="cuda") // 256
                ms = torch.rand(nb, generator=g, device="cuda") * 1e-3 * (0 if fresh else 1)
                vs = torch.rand(nb, generator=g, device="cuda") * 1e-4 * (0 if fresh else 1)
                m = (m / ms[of].clamp(min=1e-6)).clamp(-400, 400).to(torch.float8_e4m3fn)
                v = (v / vs[of].clamp(min=1e-6)).clamp(0, 50000).to(torch.float8_e5m2)
                self.ms.append(ms)
                self.vs.append(vs)
            self.m.append(m)
            self.v.append(v)
        self.lr = torch.tensor([3e-3], device="cuda")
        self.step = torch.tensor([5], dtype=torch.int32, device="cuda")
        self.gs = torch.tensor([0.7], device="cuda")
        self.wd = [0.1 * (i % 3) for i in range(len(sizes))]

    def values(self):
        """fp32 m and v as they stand."""
        out = []
        for i, n in enumerate(self.sizes):
            m, v = self.m[i].float(), self.v[i].float()
            if self.bits == 8:
                of = torch.arange(n, device="cuda") // 256
                m, v = m * self.ms[i][of], v * self.vs[i][of]
            out.append((m.cpu().numpy(), v.cpu().numpy()))
        return out

    def master(self, i):
        return self.masters[i] if self.masters[i] is not None else self.params[i]

    def run(self, B, seed=1234567890123, gs=True):
        ws = B.new_workspace(B.MOE_OP_ADAMW, 0, 0, 1, 1, 0, torch.float32)
        B.moe_adamw_step(self.params, self.grads, self.masters, self.m, self.v, self.ms, self.vs, self.wd, self.lr, self.step,
                         self.gs if gs else None, B1, B2, EPS, seed, ws)
        return B.moe_check_status(ws)


def check(B, model, seed=1234567890123):
    before = model.values()
    p0 = [np64(model.master(i)) for i in range(len(model.sizes))]
    assert model.run(B, seed) == 0
    lr, gs, step = float(model.lr), float(model.gs), int(model.step)
    for i, n in enumerate(model.sizes):
        if n == 0:
            continue
        m0, v0 = before[i]
        g = model.grads[i].float().cpu().numpy()
        wd = float(np.float32(model.wd[i]))
        want, m1, v1 = O.adamw(p0[i], g.astype(np.float64), m0.astype(np.float64), v0.astype(np.float64), lr, step, wd, B1, B2, EPS, gs)
        # m: grad_scale, two products, a sum, two rounded constants; v: the same and the square
        em = 6 * U * (np.abs(B1 * m0) + np.abs((1 - B1) * g * gs))
        ev = 8 * U * v1
        # the update: bias corrections (expm1 and its argument), root, two divisions, products: 24 roundings
        u = np.abs(want - p0[i]) + lr * wd * np.abs(p0[i])
        den = np.sqrt(v1 / (1 - B2 ** step)) + EPS
        tol = 24 * U * u + 2 * U * np.abs(p0[i]) + lr * (em / (1 - B1 ** step)) / den + 4 * U * u
        got = np64(model.master(i))
        assert (np.abs(got - want) <= tol).all(), (i, n)
        if model.dtypes[i] == torch.bfloat16:
            assert torch.equal(model.params[i], model.masters[i].to(torch.bfloat16))
        if model.bits == 32:
            assert (np.abs(np64(model.m[i]) - m1) <= em).all() and (np.abs(np64(model.v[i]) - v1) <= ev).all()
        else:
            m, v = O.adamw_states_f32(g, m0, v0, B1, B2, gs)
            cm, ms, cv, vs = O.quantize_states(m, v, O.random_words(n, i, step, seed))
            np.testing.assert_array_equal(model.ms[i].cpu().numpy(), ms)
            np.testing.assert_array_equal(model.vs[i].cpu().numpy(), vs)
            np.testing.assert_array_equal(model.m[i].float().cpu().numpy(), cm)
            np.testing.assert_array_equal(model.v[i].float().cpu().numpy(), cv)


F, H = torch.float32, torch.bfloat16


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("sizes,dtypes", [
    ([1], [F]), ([1, 2, 3, 4, 5], [H, F, H, F, H]), ([255, 256, 257], [F, H, H]), ([8192, 8191, 8193, 0, 100000], [H, F, H, F, F]),
    ([300001], [H]), ([33] * 20, [F] * 20), ([300] * 100, [H, F] * 50), ([65] * 400, [F, H] * 200)])
def test_step(B, bits, fresh, sizes, dtypes):
    check(B, Model(sizes, dtypes, bits, seed=len(sizes), fresh=fresh))


@pytest.mark.parametrize("bits", [32, 8])
def test_many_steps_follow_the_counter(B, bits):
    model = Model([1000, 77], [H, F], bits, fresh=True)
    for t in range(1, 6):
        model.step.fill_(t)
        check(B, model, seed=t * 2 ** 40 + 9)


def test_v_with_small_neighbours_stays_positive_and_the_update_bounded(B):
    model = Model([512], [F], 8, fresh=True)
    model.grads[0].fill_(1e-8)
    model.grads[0][0] = 1e4
    model.grads[0][300] = 0.0
    p0 = model.params[0].clone()
    for t in range(1, 30):
        model.step.fill_(t)
        assert model.run(B, gs=False) == 0
        if t == 1:
            model.grads[0][:256] = 0
    v = model.v[0].float()
    assert (v[1:256] > 0).all() and v[300] == 0
    # |m / sqrt(v)| of one Adam step is at most about (1 - b1) / sqrt(1 - b2) < 4, after the corrections below 8
    assert ((model.params[0] - p0).abs() <= 30 * 3e-3 * 8).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_elements_without_a_finite_gradient_stay(B, bits):
    sizes = [700, 520]
    a, b = Model(sizes, [F, H], bits), Model(sizes, [F, H], bits)
    at = [3, 255, 256, 519]
    for k, i in enumerate(at):
        a.grads[0][i] = [float("nan"), float("inf"), -float("inf"), 1e30][k]
        a.grads[1][i] = [float("nan"), float("inf"), -float("inf"), 1e30][k]
    before = a.values()
    p0 = [a.master(i).clone() for i in range(2)]
    assert a.run(B) == B.MOE_STATUS_NOT_FINITE
    b.run(B)
    for i in range(2):
        keep = torch.ones(sizes[i], dtype=torch.bool, device="cuda")
        keep[at] = False
        assert torch.equal(a.master(i)[keep], b.master(i)[keep])
        assert torch.equal(a.master(i)[at], p0[i][at])
        m, v = a.values()[i]
        if bits == 32:
            np.testing.assert_array_equal(m[at], before[i][0][at])
            np.testing.assert_array_equal(v[at], before[i][1][at])
        else:  # rounded again on the block's new scale: within a step of 1/8 (m) and 1/4 (v) or the smallest code
            assert (np.abs(m[at] - before[i][0][at]) <= np.abs(before[i][0][at]) / 8 + 2.0 ** -9 * a.ms[i].max().item()).all()
            assert (np.abs(v[at] - before[i][1][at]) <= np.abs(before[i][1][at]) / 4 + 2.0 ** -16 * a.vs[i].max().item()).all()


def test_a_step_below_one_changes_nothing(B):
    model = Model([600], [H], 8)
    model.step.zero_()
    before = [t.clone() for t in (model.params[0], model.masters[0], model.ms[0], model.vs[0])]
    codes = model.m[0].view(torch.uint8).clone()
    assert model.run(B) == B.MOE_STATUS_BAD_INDEX
    for x, y in zip(before, (model.params[0], model.masters[0], model.ms[0], model.vs[0])):
        assert torch.equal(x, y)
    assert torch.equal(codes, model.m[0].view(torch.uint8))


def test_neighbouring_memory_is_left_alone(B):
    for bits in (32, 8):
        model = Model([1027], [H], bits)
        room = torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
        p = room[:2 * 1027].view(torch.bfloat16)
        p.copy_(model.params[0])
        model.params[0] = p
        check(B, model)
        assert (room[2 * 1027:] == 7).all()


def test_captured_step_follows_lr_and_step(B):
    a, b = Model([5000], [H], 8, seed=4), Model([5000], [H], 8, seed=4)
    ws = B.new_workspace(B.MOE_OP_ADAMW, 0, 0, 1, 1, 0, torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.moe_adamw_step(a.params, a.grads, a.masters, a.m, a.v, a.ms, a.vs, a.wd, a.lr, a.step, a.gs, B1, B2, EPS, 77, ws)
    for t in (5, 6, 7):
        for model in (a, b):
            model.step.fill_(t)
            model.lr.fill_(1e-3 * t)
        g.replay()
        b.run(B, seed=77)
    torch.cuda.synchronize()
    assert torch.equal(a.masters[0], b.masters[0]) and torch.equal(a.m[0].view(torch.uint8), b.m[0].view(torch.uint8))
