"""DecodeBlock: batches of fewer tokens than it was made for, and what of the parameters it keeps."""

import gc
import weakref

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    from mixture_experts_layer_pft_gb300 import block, build

    build.build()
    return block


def params(h, f, E, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda") / s[-2] ** 0.5  # noqa: E731
    return {"gamma": torch.ones(h, device="cuda"), "Wg": rn(h, E), "bias": None, "W1": rn(E, h, f).to(dtype),
            "W3": rn(E, h, f).to(dtype), "W2": rn(E, f, h).to(dtype)}


@pytest.mark.parametrize("dtype,act8", [(torch.bfloat16, True), (torch.float32, False)])
def test_a_batch_of_fewer_tokens(block, dtype, act8):
    p = params(160, 96, 8, dtype)
    full = block.DecodeBlock(p, 20, 2, group=32, act8=act8)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(20, 160, generator=g, device="cuda").to(dtype) for _ in range(2))
    for n in (20, 13, 3, 1, 0):
        own = block.DecodeBlock(p, n, 2, group=32, act8=act8)
        want = [t.clone() for t in own.step(x[:n], r[:n])]
        got = full.step(x[:n], r[:n])
        for a, b in zip(got, want):
            assert a.shape == (n, 160) and torch.equal(a, b)
    with pytest.raises(ValueError):
        full.step(torch.cat([x, x]), torch.cat([r, r]))


def test_the_workspace_holds_any_smaller_batch(block):
    # the router of 512 tokens needs more than that of 520, and the experts' part is small
    h, f, E, T = 7168, 32, 256, 520
    g = torch.Generator(device="cuda").manual_seed(0)
    p = {"gamma": torch.ones(h, device="cuda"), "Wg": torch.randn(h, E, generator=g, device="cuda") / h ** 0.5, "bias": None}
    p.update({n: torch.zeros(E, *s, dtype=torch.bfloat16, device="cuda") for n, s in (("W1", (h, f)), ("W3", (h, f)), ("W2", (f, h)))})
    dec = block.DecodeBlock(p, T, 1)
    x = torch.randn(T, h, generator=g, device="cuda").bfloat16()
    for n in (520, 512, 257, 256, 1):
        y, s = dec.step(x[:n], x[:n])
        assert y.shape == (n, h) and (y == 0).all()


def test_full_weights_are_not_kept(block):
    p = params(64, 32, 4, torch.bfloat16)
    held = [weakref.ref(p[n]) for n in ("W1", "W3", "W2")]
    dec = block.DecodeBlock(p, 1, 2, group=32)
    p = {n: p[n] for n in ("gamma", "Wg", "bias")}
    gc.collect()
    assert all(r() is None for r in held)
    x = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")
    assert torch.isfinite(dec.step(x, x)[0].float()).all()
