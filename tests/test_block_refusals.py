"""What the operators around the layer refuse, on the CPU: every check is before any launch, and the binding refuses
tensors of another type or shape before it takes their pointers."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p(4096)   # an aligned address that no refused call reads
ODD = ctypes.c_void_p(4100)


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_pft_gb300 import binding, build

    build.build()
    binding.lib()
    return binding


def norm(B, x=P, r=P, g=P, eps=1e-6, T=4, h=16, dt=1, s=P, y=P, q=None, qs=None, rstd=P, ws=P, n=256):
    return B.lib().moe_add_rmsnorm(x, r, g, eps, T, h, dt, s, y, q, qs, rstd, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(h=0), -1), (dict(eps=-1.0), -1), (dict(dt=2), -1), (dict(h=12), -2), (dict(h=16392), -2),
    (dict(ws=None), -3), (dict(n=255), -3), (dict(x=None), -1), (dict(x=ODD), -1), (dict(g=None), -1), (dict(r=None), -1),
    (dict(s=None), -1), (dict(r=ODD), -1), (dict(s=ODD), -1), (dict(y=ODD), -1), (dict(y=None), -1), (dict(q=P), -1),
    (dict(qs=P), -1), (dict(rstd=ODD), -1), (dict(T=0, x=None, y=None), 0)])
def test_add_rmsnorm_refuses(B, kw, code):
    assert norm(B, **kw) == code


def norm_bwd(B, dy=P, s=P, g=P, rstd=P, add=P, T=4, h=16, dt=1, ds=P, dg=P, ws=P, n=1 << 20):
    return B.lib().moe_add_rmsnorm_bwd(dy, s, g, rstd, add, T, h, dt, ds, dg, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(h=4), -1), (dict(dt=-1), -1), (dict(h=20), -2), (dict(h=1 << 15), -2), (dict(ws=None), -3),
    (dict(ws=ODD), -3), (dict(n=256), -3), (dict(dg=None), -1), (dict(dy=None), -1), (dict(s=ODD), -1), (dict(g=None), -1),
    (dict(rstd=None), -1), (dict(ds=None), -1), (dict(add=ODD), -1)])
def test_add_rmsnorm_bwd_refuses(B, kw, code):
    assert norm_bwd(B, **kw) == code


def adamw(B, n=2, bits=32, numel=(8, 8), dts=(0, 0), master=(None, None), p=(P, P), scales=None, lr=P, step=P, b1=0.9,
          b2=0.99, eps=1e-8, ws=P, nbytes=256, m=(P, P), sc=P):
    k = max(n, 1)
    arr = lambda v: (ctypes.c_void_p * k)(*[(x.value if x is not None else None) for x in v][:k])  # noqa: E731
    s = arr([sc] * k) if (scales if scales is not None else bits == 8) else None
    return B.lib().moe_adamw_step(n, arr(p), arr((P, P)), arr(master), arr(m), arr((P, P)), s, s,
                                  (ctypes.c_int64 * k)(*numel[:k]), (ctypes.c_float * k)(), (ctypes.c_int32 * k)(*dts[:k]),
                                  bits, lr, step, None, b1, b2, eps, 1, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(bits=16), -1), (dict(b1=1.0), -1), (dict(b1=-0.1), -1), (dict(b2=1.0), -1), (dict(eps=0.0), -1),
    (dict(ws=None), -3), (dict(nbytes=8), -3), (dict(lr=None), -1), (dict(step=None), -1), (dict(numel=(8, -1)), -1),
    (dict(dts=(0, 3)), -1), (dict(p=(P, None)), -1), (dict(p=(P, ODD)), -1), (dict(m=(None, P)), -1),
    (dict(dts=(0, 1)), -1), (dict(dts=(0, 1), master=(None, ODD)), -1), (dict(bits=32, scales=True), -1),
    (dict(bits=8, scales=False), -1), (dict(bits=8, sc=None), -1), (dict(n=0), 0),
    ])
def test_adamw_refuses(B, kw, code):
    assert adamw(B, **kw) == code


def w4(B, x=P, xs=None, idx=P, w=P, q=P, s=P, T=2, k=2, E=4, h=64, f=64, G=64, xdt=1, dt=1, y=P, ws=P, n=1 << 20):
    return B.lib().moe_expert_ffn_w4(x, xs, idx, w, q, s, q, s, q, s, T, k, E, h, f, G, xdt, dt, y, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(k=0), -1), (dict(k=5), -1), (dict(E=1025), -1), (dict(h=0), -1), (dict(f=16), -1),
    (dict(dt=2), -1), (dict(xdt=0), -1), (dict(xdt=2), -1), (dict(xs=P), -1), (dict(xdt=2, dt=0, xs=P), -1), (dict(G=16), -1),
    (dict(G=256), -1), (dict(h=80), -2), (dict(f=72), -2), (dict(T=65537, k=1), -2), (dict(T=40000, k=2), -2),
    (dict(ws=None), -3), (dict(ws=ODD), -3), (dict(n=512), -3), (dict(x=None), -1), (dict(x=ODD), -1), (dict(idx=None), -1),
    (dict(w=None), -1), (dict(q=None), -1), (dict(s=ODD), -1), (dict(y=None), -1), (dict(T=0, x=None), 0)])
def test_expert_ffn_w4_refuses(B, kw, code):
    assert w4(B, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), -1), (dict(E=1025), -1), (dict(K=16), -1), (dict(dt=2), -1), (dict(G=48), -1), (dict(K=40), -2),
    (dict(N=36), -2), (dict(n=16), -3), (dict(W=None), -1), (dict(q=ODD), -1), (dict(s=None), -1)])
def test_quantize_w4_refuses(B, kw, code):
    a = dict(W=P, E=2, K=64, N=64, dt=1, G=32, q=P, s=P, ws=P, n=256) | kw
    assert B.lib().moe_quantize_w4(a["W"], a["E"], a["K"], a["N"], a["dt"], a["G"], a["q"], a["s"], a["ws"], a["n"], None) == code


def test_binding_refuses_other_types_and_shapes(B):
    bf, f32, f8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
    x, ws = torch.zeros(4, 16, dtype=bf), torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):  # not on a CUDA device
        B.moe_add_rmsnorm(x, None, torch.ones(16), 1e-6, None, x.clone(), None, None, None, ws)
    meta = lambda *s, dtype=f32: torch.empty(*s, dtype=dtype)  # noqa: E731
    for bad in (dict(params=[meta(8)], grads=[meta(8, dtype=bf)]), dict(params=[meta(8)], grads=[]),
                dict(params=[meta(8)], grads=[meta(9)])):
        with pytest.raises(ValueError):
            B.moe_adamw_step(bad["params"], bad["grads"], None, [meta(8)], [meta(8)], None, None, 0.0, meta(1),
                             meta(1, dtype=torch.int32), None, 0.9, 0.99, 1e-8, 0, ws)
    with pytest.raises(TypeError):
        B.moe_adamw_step([meta(8, dtype=torch.float16)], [meta(8, dtype=torch.float16)], None, [meta(8)], [meta(8)], None, None,
                         0.0, meta(1), meta(1, dtype=torch.int32), None, 0.9, 0.99, 1e-8, 0, ws)
    with pytest.raises(ValueError):
        B._check(meta(4, 2), "q_scale", f32, (4, 1))
    with pytest.raises(ValueError):
        B._check(meta(4, 2, dtype=f8), "y", bf, (4, 2))


def test_tensors_without_an_address_raise_and_do_not_end_the_process(B):
    sparse = torch.zeros(4, 4).to_sparse()
    nested = torch.nested.nested_tensor([torch.zeros(2), torch.zeros(3)])
    for t in (sparse, nested, torch.empty(4, 4, device="meta"), torch.zeros(4, 4).t()):
        with pytest.raises(ValueError):
            B._check(t, "x", torch.float32, (4, 4))
    with pytest.raises((TypeError, ValueError)):
        B._check("no tensor", "x", torch.float32, (4, 4))
    one = torch.zeros(8)
    for wd in ([0.1, 0.2], []):
        with pytest.raises(ValueError):
            B.moe_adamw_step([one], [one], None, [one], [one], None, None, wd, one[:1], torch.ones(1, dtype=torch.int32), None, 0.9,
                             0.99, 1e-8, 0, torch.zeros(256, dtype=torch.uint8))
    for bad in ([sparse], [nested], ["x"], 3):
        with pytest.raises((TypeError, ValueError)):
            B.moe_adamw_step(bad, bad, None, bad, bad, None, None, 0.1, one[:1], torch.ones(1, dtype=torch.int32), None, 0.9, 0.99,
                             1e-8, 0, torch.zeros(256, dtype=torch.uint8))


def test_workspace_sizes(B):
    bf = torch.bfloat16
    for op in (B.MOE_OP_ADD_RMSNORM, B.MOE_OP_ADAMW):
        assert B.workspace_size(op, 4096, 7168, 256, 8, 2048, bf) == 256
    assert B.workspace_size(B.MOE_OP_EXPERT_FFN_W4, 5, 64, 8, 2, 96, bf) >= 256 + 10 * 96 * 2 + 10 * 64 * 4
    assert B.workspace_size(B.MOE_OP_ADD_RMSNORM_BWD, 1, 7168, 1, 1, 0, bf) % 256 == 0
