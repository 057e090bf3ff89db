"""What the operators around the MoE layer are measured on: the add + RMSNorm before it (with its backward and an
8-bit output), the AdamW step on its parameters (states in 32 or 8 bits), and its experts over 4-bit weights for the few
tokens of a decode step.

Sizes are those of ``workloads.WORKLOADS``'s layers (Small h=2048 f=1408 E=64 k=6, Medium h=5120 f=1536 E=128 k=6, Large
h=7168 f=2048 E=256 k=8, the long-sequence fp32 layer h=2048 f=2048 E=128 k=2, the tiny one h=128 f=64 E=8 k=2) and odd
ones beside them.  ``run`` computes a case in elementary torch operations, or with ``own`` by the framework's calls.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6
Q_GROUP = 128      # columns of one scale of the norm's 8-bit output
BLOCK = 256        # elements of one scale of the 8-bit optimizer states
BETA1, BETA2, ADAM_EPS, DECAY = 0.9, 0.999, 1e-8, 0.1
M32 = 0xFFFFFFFF


def listed():
    return [
        # one token of a decode step enters the Large layer: the residual's addition, y for the router, 8 bits for the experts
        {"name": "norm-decode-q8", "op": "norm", "T": 1, "h": 7168, "dtype": "bf16", "residual": True, "q8": True},
        # a training batch of the Large layer, with the 8-bit output beside y
        {"name": "norm-large-q8", "op": "norm", "T": 4096, "h": 7168, "dtype": "bf16", "residual": True, "q8": True},
        # its backward, with the gradient that comes down the residual stream
        {"name": "norm-bwd-large", "op": "norm_bwd", "T": 4096, "h": 7168, "dtype": "bf16", "residual": True},
        # a ragged batch in fp32 with a width that is no multiple of 128, first norm of a model (no residual gradient)
        {"name": "norm-bwd-odd-fp32", "op": "norm_bwd", "T": 1533, "h": 1000, "dtype": "f32", "residual": False},
        # all parameters of the tiny fp32 layer: latency
        {"name": "adamw32-tiny", "op": "adamw", "layer": "128,64,8,1", "dtype": "f32", "bits": 32, "ragged": 0},
        # all parameters of the Small layer (554 M) with 32-bit states
        {"name": "adamw32-small", "op": "adamw", "layer": "2048,1408,64,1", "dtype": "bf16", "bits": 32, "ragged": 0},
        # the same with 8-bit states
        {"name": "adamw8-small", "op": "adamw", "layer": "2048,1408,64,1", "dtype": "bf16", "bits": 8, "ragged": 0},
        # many small tensors of odd sizes: four narrow layers, with biases that are no multiple of anything
        {"name": "adamw8-ragged", "op": "adamw", "layer": "264,88,16,4", "dtype": "bf16", "bits": 8, "ragged": 37},
        # one token through the Small layer's experts
        {"name": "w4-decode-small", "op": "w4", "T": 1, "h": 2048, "f": 1408, "E": 64, "k": 6, "group": 128,
         "x": "bf16", "skew": False},
        # one token through the Large layer's experts, in the norm's 8 bits
        {"name": "w4-decode-large-q8", "op": "w4", "T": 1, "h": 7168, "f": 2048, "E": 256, "k": 8, "group": 128,
         "x": "q8", "skew": False},
        # a decode batch of 64 sequences through the Medium layer with its skewed router
        {"name": "w4-batch-medium", "op": "w4", "T": 64, "h": 5120, "f": 1536, "E": 128, "k": 6, "group": 128,
         "x": "bf16", "skew": True},
        # an odd batch in fp32 through the long-sequence layer, finer groups
        {"name": "w4-batch-fp32", "op": "w4", "T": 13, "h": 2048, "f": 2048, "E": 128, "k": 2, "group": 32,
         "x": "f32", "skew": True},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "adamw", "adamw", "w4", "w4", "w4"])
    if op in ("norm", "norm_bwd"):
        h = _log(rng, 64, 8192, 8)
        T = _log(rng, 1, min(16384, 4096 * 7168 // h))
        case = {"op": op, "T": T, "h": h, "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.7}
        if op == "norm":
            case["q8"] = rng.random() < 0.5
        return case
    if op == "adamw":
        h, f, E = _log(rng, 64, 2048, 8), _log(rng, 64, 1408, 8), _log(rng, 2, 64)
        return {"op": op, "layer": "%d,%d,%d,%d" % (h, f, E, rng.choice([1, 1, 2, 3])), "dtype": rng.choice(["bf16", "f32"]),
                "bits": rng.choice([8, 32]), "ragged": rng.choice([0, 5, 37])} if h * f * E < 60e6 else draw(rng)
    E = rng.choice([8, 16, 33, 64, 96, 128])
    h, f = _log(rng, 128, 5120, 32), _log(rng, 64, 2048, 32)
    if E * h * f > 5e8:
        return draw(rng)
    return {"op": op, "T": _log(rng, 1, 64), "h": h, "f": f, "E": E, "k": rng.choice([1, 2, 4, 6, 8]),
            "group": rng.choice([32, 64, 128, 128]), "x": rng.choice(["bf16", "bf16", "q8", "f32"]), "skew": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _stream_rows(gen, T, h, dtype):
    """Rows of a residual stream: a few channels much larger than the others."""
    x = _randn(gen, T, h)
    x[:, :: 97] *= 8.0
    return x.to(dtype)


def _gamma(gen, h):
    return 1.0 + 0.1 * torch.randn(h, generator=gen, device="cuda")


def _workspace(op, T, h, E, k, f, dtype):
    """The framework's workspace, which a program keeps; the plain form needs none."""
    if not own:
        return None
    from mixture_experts_layer_pft_gb300 import binding as B

    return B.new_workspace(getattr(B, op), T, h, E, k, f, dtype)


def _prepare_norm(case, seed):
    gen, T, h, dt = _gen(seed), case["T"], case["h"], _dtype(case["dtype"])
    s = {"x": _stream_rows(gen, T, h, dt), "gamma": _gamma(gen, h),
         "residual": _randn(gen, T, h, std=2.0, dtype=dt) if case["residual"] else None}
    s["s"] = torch.empty(T, h, dtype=dt, device="cuda") if case["residual"] else None
    s["y"] = torch.empty(T, h, dtype=dt, device="cuda")
    s["rstd"] = torch.empty(T, device="cuda")
    s["q"] = torch.empty(T, h, dtype=torch.float8_e4m3fn, device="cuda") if case["q8"] else None
    s["q_scale"] = torch.empty(T, -(-h // Q_GROUP), device="cuda") if case["q8"] else None
    s["ws"] = _workspace("MOE_OP_ADD_RMSNORM", T, h, 1, 1, 0, dt)
    return s


def _prepare_norm_bwd(case, seed):
    gen, T, h, dt = _gen(seed), case["T"], case["h"], _dtype(case["dtype"])
    s = {"s": _stream_rows(gen, T, h, dt), "gamma": _gamma(gen, h), "dy": _randn(gen, T, h, dtype=dt),
         "ds_add": _randn(gen, T, h, dtype=dt) if case["residual"] else None}
    s["rstd"] = (s["s"].double().square().mean(1) + EPS).rsqrt().float()  # as the forward left it
    s["ds"] = torch.empty(T, h, dtype=dt, device="cuda")
    s["dgamma"] = torch.empty(h, device="cuda")
    s["ws"] = _workspace("MOE_OP_ADD_RMSNORM_BWD", T, h, 1, 1, 0, dt)
    return s


def _tensor_sizes(case):
    """{dtype: sizes of its tensors}: per layer W_g and the norm's weight in fp32, the three expert weights in the layer's
    type, and `ragged` biases of odd sizes."""
    h, f, E, layers = (int(v) for v in case["layer"].split(","))
    sizes = {"f32": [h * E, h] * layers + [17 + 61 * i for i in range(case["ragged"])]}
    sizes.setdefault(case["dtype"], []).extend([E * h * f] * 3 * layers)
    return sizes


def _prepare_adamw(case, seed):
    """Parameters, gradients and states as flat buffers of each type, a tensor beginning at each multiple of BLOCK, and the
    lists of tensors (views) that a program has."""
    gen, groups = _gen(seed), []
    for name, sizes in _tensor_sizes(case).items():
        padded = [-(-n // BLOCK) * BLOCK for n in sizes]
        starts = np.concatenate([[0], np.cumsum(padded)])
        total, blocks = int(starts[-1]), int(starts[-1]) // BLOCK
        used = torch.zeros(blocks, dtype=torch.int64)  # elements in use of each block
        for a, n, m in zip(starts, sizes, padded):
            used[a // BLOCK:(a + m) // BLOCK] = BLOCK
            used[(a + m) // BLOCK - 1] = n - (m - BLOCK)
        inside = (torch.arange(BLOCK, device="cuda") < used.cuda()[:, None]).view(-1)
        size = torch.exp(_randn(gen, blocks, 1) - 7.0).expand(blocks, BLOCK).reshape(-1)  # gradients of other sizes in each block
        p = _randn(gen, total, std=0.02).mul_(inside)
        g = _randn(gen, total).mul_(size).mul_(inside)
        m = _randn(gen, total, std=0.3).mul_(size).mul_(inside)
        v = _randn(gen, total).square_().mul_(0.5).add_(0.5).mul_(size).mul_(size).mul_(inside)
        grp = {"dtype": name, "sizes": sizes, "starts": [int(a) for a in starts[:-1]], "master": p, "p": p, "m": m, "v": v,
               "g": g.to(_dtype(name)), "ms": None, "vs": None}
        if name == "bf16":
            grp["p"] = p.to(torch.bfloat16)
        if case["bits"] == 8:
            mb, vb = m.view(blocks, BLOCK), v.view(blocks, BLOCK)
            grp["ms"] = mb.abs().amax(1) / 256.0
            grp["vs"] = vb.amax(1) / 32768.0
            grp["m"] = (mb / grp["ms"][:, None]).to(torch.float8_e4m3fn).view(-1)
            grp["v"] = (vb / grp["vs"][:, None]).clamp(min=2.0 ** -16).mul_(inside.view(blocks, BLOCK)).to(torch.float8_e5m2).view(-1)
        groups.append(grp)
    s = {"groups": groups, "lr": torch.tensor([2e-4], device="cuda"), "step": torch.tensor([37], dtype=torch.int32, device="cuda"),
         "grad_scale": torch.tensor([0.5], device="cuda"), "seed": seed * 1000003 + 17, "bits": case["bits"]}
    views = lambda key: [grp[key][a:a + n] for grp in groups for a, n in zip(grp["starts"], grp["sizes"])]  # noqa: E731
    scales = lambda key: [grp[key][a // BLOCK:a // BLOCK + -(-n // BLOCK)] for grp in groups  # noqa: E731
                          for a, n in zip(grp["starts"], grp["sizes"])] if case["bits"] == 8 else None
    s["params"], s["grads"], s["m"], s["v"] = views("p"), views("g"), views("m"), views("v")
    s["masters"] = [grp["master"][a:a + n] if grp["dtype"] == "bf16" else None for grp in groups
                    for a, n in zip(grp["starts"], grp["sizes"])]
    s["m_scale"], s["v_scale"] = scales("ms"), scales("vs")
    s["ws"] = _workspace("MOE_OP_ADAMW", 0, 0, 1, 1, 0, torch.float32)
    return s


def _routing(case, seed):
    """top-k experts and softmax weights of each token, from N(0,1) logits, with the Zipf-like bias where `skew`."""
    r = np.random.RandomState(seed % (1 << 31))
    T, E, k = case["T"], case["E"], case["k"]
    logits = r.standard_normal((T, E))
    if case["skew"]:
        logits = logits - 1.6 * np.log(np.arange(E) + 1.0)
    p = np.exp(logits - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    return idx.astype(np.int32), np.take_along_axis(p, idx, 1).astype(np.float32)


def _quantized(gen, E, K, N, group):
    """N(0, 1/K) weights of E experts in 4 bits: [E, N, K/2] bytes (input 2i in the low half of byte i, 2i+1 in the high one,
    offset by 8) and a bf16 scale for each `group` inputs of an output, [E, N, ceil(K/group)]."""
    n = -(-K // group)
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(E, N, n, dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 26) // (K * N))
    for e in range(0, E, step):
        m = min(step, E - e)
        w = torch.randn(m, N, K, generator=gen, device="cuda") / math.sqrt(K)
        w = torch.nn.functional.pad(w, (0, n * group - K)).view(m, N, n, group)
        s = (w.abs().amax(3) / 7.0).to(torch.bfloat16)
        c = (w / s.float().clamp(min=1e-30)[..., None]).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
        c = c.view(m, N, n * group)[:, :, :K]
        q[e:e + m] = c[:, :, 0::2] | (c[:, :, 1::2] << 4)
        scale[e:e + m] = s
    return q, scale


def _prepare_w4(case, seed):
    gen, T, h, f, E = _gen(seed), case["T"], case["h"], case["f"], case["E"]
    dt = torch.float32 if case["x"] == "f32" else torch.bfloat16
    idx, w = _routing(case, seed)
    s = {"group": case["group"], "dtype": dt, "topk_idx": torch.from_numpy(idx).cuda(), "topk_w": torch.from_numpy(w).cuda()}
    x = _randn(gen, T, h)
    s["x_scale"] = None
    if case["x"] == "q8":
        s["x"], s["x_scale"] = _quantize_rows(x)
    else:
        s["x"] = x.to(dt)
    s["W1q"], s["W1s"] = _quantized(gen, E, h, f, case["group"])
    s["W3q"], s["W3s"] = _quantized(gen, E, h, f, case["group"])
    s["W2q"], s["W2s"] = _quantized(gen, E, f, h, case["group"])
    s["y"] = torch.empty(T, h, dtype=dt, device="cuda")
    s["ws"] = _workspace("MOE_OP_EXPERT_FFN_W4", T, h, E, case["k"], f, dt)
    return s


def prepare(case, seed):
    state = {"norm": _prepare_norm, "norm_bwd": _prepare_norm_bwd, "adamw": _prepare_adamw, "w4": _prepare_w4}[case["op"]](case, seed)
    state["op"] = case["op"]
    return state


# ------------------------------------------------------------------------------------------------ the plain forms


def _quantize_rows(v):
    """fp32 rows in e4m3, with an fp32 scale for each Q_GROUP columns: amax / 448."""
    T, h = v.shape
    n = -(-h // Q_GROUP)
    g = torch.nn.functional.pad(v, (0, n * Q_GROUP - h)).view(T, n, Q_GROUP)
    scale = g.abs().amax(2).clamp(min=2.0 ** -100) / 448.0
    q = (g / scale[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(T, n * Q_GROUP)[:, :h].contiguous(), scale


def _plain_norm(s):
    rows = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    r = rows.float()
    rstd = (r.square().mean(1) + EPS).rsqrt()
    v = r * rstd[:, None] * s["gamma"]
    out = {"y": v.to(rows.dtype), "rstd": rstd}
    if s["residual"] is not None:
        out["s"] = rows
    if s["q"] is not None:
        out["q"], out["q_scale"] = _quantize_rows(v)
    return out


def _plain_norm_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh, g = s["s"].float() * rstd, dy * s["gamma"]
    ds = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["ds_add"] is not None:
        ds = ds + s["ds_add"].float()
    return {"ds": ds.to(s["s"].dtype), "dgamma": (dy * xh).sum(0)}


def _philox(c0, c1, c2, c3, seed):
    """Philox4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, 2011) on int64 tensors that hold 32-bit words."""
    k0, k1 = seed & M32, (seed >> 32) & M32
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return c0, c1, c2, c3


def _random_bits(grp, first, step, seed):
    """32 random bits for each element of the flat buffer: four elements share a Philox call whose counter is the number of
    the four in their tensor, the tensor's number and the step."""
    dev = grp["p"].device
    blocks = torch.tensor([-(-n // BLOCK) for n in grp["sizes"]], device=dev)
    tensor = torch.repeat_interleave(torch.arange(len(grp["sizes"]), device=dev), blocks)
    local = torch.arange(tensor.numel(), device=dev) - (blocks.cumsum(0) - blocks)[tensor]
    four = local[:, None] * (BLOCK // 4) + torch.arange(BLOCK // 4, device=dev)
    zero = torch.zeros_like(four)
    words = _philox(four & M32, four >> 32, zero + (tensor + first)[:, None], zero + step.long(), seed)
    return torch.stack(words, 2).view(-1, BLOCK)


def _round_up_or_down(x, bits16, drop, low):
    """fp32 x >= 0 rounded to 23 - drop mantissa bits, up with the probability of what is cut off; below `low` (a power of two)
    on the grid of [low, 2 low)."""
    small = x < low
    t = torch.where(small, x + low, x).view(torch.int32)
    t = (t + ((bits16 << (drop - 16)) | (1 << (drop - 17))).int()) & -(1 << drop)
    t = t.view(torch.float32)
    return torch.where(small, t - low, t)


def _plain_adamw(s):
    step, lr, out, first = s["step"], s["lr"], [], 0
    bc1 = (-torch.expm1(step.double() * math.log(BETA1))).float()
    bc2 = (-torch.expm1(step.double() * math.log(BETA2))).float()
    for grp in s["groups"]:
        g = grp["g"].float() * s["grad_scale"]
        m, v = grp["m"].float(), grp["v"].float()
        if s["bits"] == 8:
            m = (m.view(-1, BLOCK) * grp["ms"][:, None]).view(-1)
            v = (v.view(-1, BLOCK) * grp["vs"][:, None]).view(-1)
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + (g * g) * (1 - BETA2)
        p = grp["master"]
        p = p - lr * (DECAY * p + (m / bc1) / ((v / bc2).sqrt() + ADAM_EPS))
        grp["master"].copy_(p)
        if grp["dtype"] == "bf16":
            grp["p"].copy_(p)
        if s["bits"] == 8:
            bits = _random_bits(grp, first, step, s["seed"])
            mb, vb = m.view(-1, BLOCK), v.view(-1, BLOCK)
            ms = mb.abs().amax(1).clamp(min=2.0 ** -100) * 2.0 ** -8
            vs = vb.amax(1).clamp(min=2.0 ** -100) * 2.0 ** -15
            mq = _round_up_or_down(mb.abs() * ms.reciprocal()[:, None], bits & 0xFFFF, 20, 2.0 ** -6)
            vq = _round_up_or_down(vb * vs.reciprocal()[:, None], bits >> 16, 21, 2.0 ** -14)
            vq = torch.where((vq == 0) & (vb > 0), 2.0 ** -16, vq)
            grp["m"].copy_(torch.copysign(mq, mb).view(-1).to(torch.float8_e4m3fn))
            grp["v"].copy_(vq.view(-1).to(torch.float8_e5m2))
            grp["ms"].copy_(ms)
            grp["vs"].copy_(vs)
        else:
            grp["m"].copy_(m)
            grp["v"].copy_(v)
        first += len(grp["sizes"])
        out.append(_adamw_out(grp))
    return out


def _adamw_out(grp):
    return {key: grp[key] for key in ("p", "master", "m", "v", "ms", "vs") if grp[key] is not None and (key != "master" or grp["dtype"] == "bf16")}


def _weights(q, scale, group):
    """[..., N, K] fp32 from 4 bits."""
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).float() - 8.0
    return c * scale.float().repeat_interleave(group, -1)[..., :c.shape[-1]]


def _plain_w4(s):
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].repeat_interleave(Q_GROUP, 1)[:, :x.shape[1]]
    idx, (T, k), G = s["topk_idx"].long(), s["topk_idx"].shape, s["group"]
    if T * k <= s["W1q"].shape[0]:  # the weights of each row's expert
        e, rows = idx.view(-1), x.repeat_interleave(k, 0)[:, :, None]
        a = torch.bmm(_weights(s["W1q"][e], s["W1s"][e], G), rows)
        a = a * torch.sigmoid(a) * torch.bmm(_weights(s["W3q"][e], s["W3s"][e], G), rows)
        y = torch.bmm(_weights(s["W2q"][e], s["W2s"][e], G), a).view(T, k, -1)
    else:  # all experts on all tokens, and each token's k of them
        a = torch.matmul(_weights(s["W1q"], s["W1s"], G), x.t())
        a = a * torch.sigmoid(a) * torch.matmul(_weights(s["W3q"], s["W3s"], G), x.t())
        y = torch.bmm(_weights(s["W2q"], s["W2s"], G), a).permute(2, 0, 1)
        y = torch.gather(y, 1, idx[:, :, None].expand(-1, -1, y.shape[2]))
    return (y * s["topk_w"][:, :, None]).sum(1).to(s["dtype"])


# ------------------------------------------------------------------------------------------------ one pass


def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "adamw": _plain_adamw, "w4": _plain_w4}[s["op"]](s)
    from mixture_experts_layer_pft_gb300 import binding as B

    if s["op"] == "norm":
        B.moe_add_rmsnorm(s["x"], s["residual"], s["gamma"], EPS, s["s"], s["y"], s["q"], s["q_scale"], s["rstd"], s["ws"])
        return {key: s[key] for key in ("y", "rstd", "s", "q", "q_scale") if s[key] is not None}
    if s["op"] == "norm_bwd":
        B.moe_add_rmsnorm_bwd(s["dy"], s["s"], s["gamma"], s["rstd"], s["ds_add"], s["ds"], s["dgamma"], s["ws"])
        return {"ds": s["ds"], "dgamma": s["dgamma"]}
    if s["op"] == "adamw":
        B.moe_adamw_step(s["params"], s["grads"], s["masters"], s["m"], s["v"], s["m_scale"], s["v_scale"], DECAY, s["lr"],
                         s["step"], s["grad_scale"], BETA1, BETA2, ADAM_EPS, s["seed"], s["ws"])
        return [_adamw_out(grp) for grp in s["groups"]]
    B.moe_expert_ffn_w4(s["x"], s["x_scale"], s["topk_idx"], s["topk_w"], s["W1q"], s["W1s"], s["W3q"], s["W3s"], s["W2q"], s["W2s"],
                        s["group"], s["y"], s["ws"])
    return s["y"]


def work(case):
    if case["op"] in ("norm", "norm_bwd"):
        T, h, es = case["T"], case["h"], 4 if case["dtype"] == "f32" else 2
        if case["op"] == "norm_bwd":
            return {"bytes": T * h * es * (4 if case["residual"] else 3) + 4 * T + 8 * h, "flops": 9 * T * h}
        b = T * h * es * (4 if case["residual"] else 2) + 4 * T + 4 * h
        return {"bytes": b + (T * h + 4 * T * -(-h // Q_GROUP) if case["q8"] else 0), "flops": (8 if case["q8"] else 5) * T * h}
    if case["op"] == "adamw":
        # read and written: the fp32 value and both states; read: the gradient; written: the bf16 copy
        state = 2 * 2 * (4 if case["bits"] == 32 else 1 + 4 / BLOCK)
        n = {name: sum(sizes) for name, sizes in _tensor_sizes(case).items()}
        return {"bytes": sum(c * (8 + state + 4) for c in n.values()), "flops": 15 * sum(n.values())}
    T, h, f, k = case["T"], case["h"], case["f"], case["k"]
    active = len(np.unique(_routing(case, 1)[0]))
    groups = 2 * f * -(-h // case["group"]) + h * -(-f // case["group"])
    rows = T * h * ({"bf16": 2, "f32": 4, "q8": 1}[case["x"]] + (4 if case["x"] == "f32" else 2))
    return {"bytes": active * (1.5 * h * f + 2 * groups) + rows + 8 * T * k, "flops": 6 * T * k * h * f}


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits


def _exact_groups(v):
    """(codes, scales) of the 8-bit output, by the table of e4m3 values."""
    T, h = v.shape
    n = -(-h // Q_GROUP)
    scale = torch.stack([v[:, i * Q_GROUP:(i + 1) * Q_GROUP].abs().amax(1) for i in range(n)], 1).clamp(min=2.0 ** -100) / 448
    u = v / scale.repeat_interleave(Q_GROUP, 1)[:, :h]
    e = torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6)))
    grid = torch.exp2(e - 3)
    return (torch.round(u / grid) * grid).clamp(-448, 448), scale


def _exact_norm(s):
    a = s["x"].double()
    if s["residual"] is not None:
        a = (a + s["residual"].double()).to(s["x"].dtype).double()  # s itself is an output that the norm reads
    rstd = 1 / torch.sqrt((a * a).sum(1) / a.shape[1] + EPS)
    v = torch.einsum("th,t,h->th", a, rstd, s["gamma"].double())
    out = {"y": v, "rstd": rstd}
    if s["residual"] is not None:
        out["s"] = a
    if s["q"] is not None:
        out["q"], out["q_scale"] = _exact_groups(v)
    return out


def _exact_norm_bwd(s):
    dy, a, r, gamma = s["dy"].double(), s["s"].double(), s["rstd"].double(), s["gamma"].double()
    inner = torch.einsum("th,th,h->t", dy, a, gamma) * r ** 3 / a.shape[1]
    ds = dy * gamma * r[:, None] - a * inner[:, None]
    if s["ds_add"] is not None:
        ds += s["ds_add"].double()
    return {"ds": ds, "dgamma": torch.einsum("th,th,t->h", dy, a, r)}


def _exact_words(n, tensor, step, seed):
    """Philox4x32-7 words of a tensor of n elements, with products in 16-bit halves."""
    c = torch.arange(-(-n // 4), device="cuda")
    x = [c % 2 ** 32, c // 2 ** 32, torch.full_like(c, tensor), torch.full_like(c, step)]
    key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]

    def product(v, by):
        lo, hi = v * (by % 65536), v * (by // 65536)  # both below 2^48
        mid = hi % 65536 * 65536 + lo                 # below 2^49
        return hi // 65536 + mid // 2 ** 32, mid % 2 ** 32

    for _ in range(7):
        h0, l0 = product(x[0], 0xD2511F53)
        h1, l1 = product(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return torch.stack(x, 1).reshape(-1)[:n]


def _exact_codes(x, random16, mantissa, smallest):
    """x >= 0 on the grid of an 8-bit float with `mantissa` bits and smallest normal exponent `smallest`, up where the 16 random
    bits say so."""
    grid = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** smallest))) - mantissa)
    return torch.floor(x / grid + (random16.double() + 0.5) / 65536) * grid


def _exact_adamw(s):
    out, number = [], 0
    t, lr, scale = int(s["step"]), float(s["lr"]), float(s["grad_scale"])
    for grp in s["groups"]:
        got = {key: torch.zeros(grp["p"].numel(), dtype=torch.float64, device="cuda") for key in ("p", "m", "v")}
        if s["bits"] == 8:
            got["ms"] = torch.zeros(grp["ms"].numel(), dtype=torch.float64, device="cuda")
            got["vs"] = torch.zeros_like(got["ms"])
        for a, n in zip(grp["starts"], grp["sizes"]):
            g = grp["g"][a:a + n].double() * scale
            m, v = grp["m"][a:a + n].to(torch.float32).double(), grp["v"][a:a + n].to(torch.float32).double()
            b, nb = a // BLOCK, -(-n // BLOCK)
            if s["bits"] == 8:
                of = torch.arange(n, device="cuda") // BLOCK
                m, v = m * grp["ms"][b:b + nb].double()[of], v * grp["vs"][b:b + nb].double()[of]
            m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
            p = grp["master"][a:a + n].double()
            got["p"][a:a + n] = p * (1 - lr * DECAY) - lr * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + ADAM_EPS)
            if s["bits"] == 8:
                words = _exact_words(n, number, t, s["seed"])
                most = lambda u: torch.nn.functional.pad(u, (0, nb * BLOCK - n)).view(nb, BLOCK).amax(1).clamp(min=2.0 ** -100)  # noqa: E731
                ms, vs = most(m.abs()) / 256, most(v) / 32768
                got["ms"][b:b + nb], got["vs"][b:b + nb] = ms, vs
                got["m"][a:a + n] = torch.sign(m) * _exact_codes(m.abs() / ms[of], words % 65536, 3, -6)
                code = _exact_codes(v / vs[of], words // 65536, 2, -14)
                got["v"][a:a + n] = torch.where(v > 0, code.clamp(min=2.0 ** -16), code)
            else:
                got["m"][a:a + n], got["v"][a:a + n] = m, v
            number += 1
        if s["bits"] == 8:  # blocks are whole tensors' own: none is left out
            assert bool((got["ms"] > 0).all())
        if grp["dtype"] == "bf16":
            got["master"] = got["p"]
        out.append(got)
    return out


def _exact_w4(s, case):
    T, k, h, f, G = case["T"], case["k"], case["h"], case["f"], case["group"]
    x = s["x"].to(torch.float32).double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double()[:, torch.arange(h, device="cuda") // Q_GROUP]

    def matrix(q, scale, e, K):
        w = torch.empty(q.shape[1], K, dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (q[e] % 16).double() - 8, (q[e] // 16).double() - 8
        return w * scale[e].double()[:, torch.arange(K, device="cuda") // G]

    y = torch.zeros(T, h, dtype=torch.float64, device="cuda")
    idx = s["topk_idx"].cpu().numpy()
    for e in np.unique(idx):
        t, j = (torch.from_numpy(v).cuda() for v in np.nonzero(idx == e))
        z = x[t] @ matrix(s["W1q"], s["W1s"], e, h).t()
        a = z / (1 + torch.exp(-z)) * (x[t] @ matrix(s["W3q"], s["W3s"], e, h).t())
        y.index_add_(0, t, s["topk_w"].double()[t, j][:, None] * (a @ matrix(s["W2q"], s["W2s"], e, f).t()))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w4":
        return _exact_w4(s, case)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "adamw": _exact_adamw}[case["op"]](s)
