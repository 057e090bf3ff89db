"""The pre-norm MoE block around the layer: its training step with the optimizer, and its decode step in 4 bits.

    s = x + residual;  n = RMSNorm(s) * gamma;  y = MoE(n);  the stream goes on as s + y

The addition of y is the next block's (its x is this block's y, its residual this block's s), so every add happens inside
a norm.  ``BlockBuffers`` owns what a training step writes, ``block_forward`` and ``block_backward`` issue its calls,
``AdamW`` updates the parameters in place, and ``DecodeBlock`` serves a few tokens from quantised experts.  All arithmetic
is the library's; PyTorch owns the memory.
"""

from __future__ import annotations

import torch

from . import binding as B
from . import layer


class BlockBuffers:
    """Device buffers of one block's training step: the layer's, and the norm's on both sides of it."""

    def __init__(self, T: int, h: int, E: int, k: int, f: int, dtype: torch.dtype, device="cuda", eps: float = 1e-6, **kw):
        self.layer = layer.LayerBuffers(T, h, E, k, f, dtype, device, **kw)
        self.eps = eps
        self.s = torch.empty(T, h, dtype=dtype, device=device)
        self.n = torch.empty(T, h, dtype=dtype, device=device)
        self.rstd = torch.empty(T, dtype=torch.float32, device=device)
        self.ws = B.new_workspace(B.MOE_OP_ADD_RMSNORM_BWD, T, h, 1, 1, 0, dtype, device)
        if self.layer.backward:
            self.ds = torch.empty(T, h, dtype=dtype, device=device)
            self.dgamma = torch.empty(h, dtype=torch.float32, device=device)


def block_forward(params: dict, x: torch.Tensor, residual: torch.Tensor, b: BlockBuffers):
    """Returns (y, s).  ``params``: gamma [h] fp32 and the layer's Wg, bias (or none), W1, W3, W2."""
    B.moe_add_rmsnorm(x, residual, params["gamma"], b.eps, b.s, b.n, None, None, b.rstd, b.ws)
    layer.forward(dict(params, x=b.n), b.layer)
    return b.layer.y, b.s


def block_backward(params: dict, dy: torch.Tensor, ds: torch.Tensor, b: BlockBuffers):
    """From the gradients of y and s: the gradient of x and of residual (b.ds), and the parameters' in b."""
    layer.backward(dict(params, x=b.n), dy, b.layer)
    B.moe_add_rmsnorm_bwd(b.layer.dx, b.s, params["gamma"], b.rstd, ds, b.ds, b.dgamma, b.ws)
    return b.ds


def parameters(params: dict, b: BlockBuffers):
    """(parameters, gradients) of a block, in one order."""
    lb = b.layer
    return ([params[n] for n in ("gamma", "Wg", "W1", "W3", "W2")], [b.dgamma, lb.dWg, lb.dW1, lb.dW3, lb.dW2])


class AdamW:
    """AdamW over lists of tensors, with states in 32 or 8 bits.

    bf16 parameters get an fp32 master, made from them here.  ``weight_decay`` is a number or one per tensor.  ``step``
    counts on the device, as lr lives there: a captured step follows both.  The kernel marks a gradient that is not finite
    (and skips its element) in the status word of ``ws``."""

    def __init__(self, params, grads, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01, bits: int = 32,
                 seed: int = 0):
        if bits not in (32, 8):
            raise ValueError("states have 32 or 8 bits")
        dev = params[0].device
        self.params, self.grads = list(params), list(grads)
        self.masters = [p.float() if p.dtype == torch.bfloat16 else None for p in params]
        self.betas, self.eps, self.weight_decay, self.seed = betas, eps, weight_decay, seed
        self.lr = torch.tensor([lr], dtype=torch.float32, device=dev)
        self.step_count = torch.zeros(1, dtype=torch.int32, device=dev)
        types = (torch.float32, torch.float32) if bits == 32 else (torch.float8_e4m3fn, torch.float8_e5m2)
        self.m = [torch.zeros(p.shape, dtype=types[0], device=dev) for p in params]
        self.v = [torch.zeros(p.shape, dtype=types[1], device=dev) for p in params]
        blocks = lambda p: torch.zeros(-(-p.numel() // 256), dtype=torch.float32, device=dev)  # noqa: E731
        self.m_scale = [blocks(p) for p in params] if bits == 8 else None
        self.v_scale = [blocks(p) for p in params] if bits == 8 else None
        self.ws = B.new_workspace(B.MOE_OP_ADAMW, 0, 0, 1, 1, 0, torch.float32, dev)

    def step(self, grad_scale: torch.Tensor | None = None):
        """One step on the current stream; ``grad_scale`` (fp32[1] on the device) multiplies every gradient."""
        self.step_count.add_(1)
        try:
            B.moe_adamw_step(self.params, self.grads, self.masters, self.m, self.v, self.m_scale, self.v_scale, self.weight_decay,
                             self.lr, self.step_count, grad_scale, *self.betas, self.eps, self.seed, self.ws)
        except (TypeError, ValueError, B.MoEError):  # refused: no step was made
            self.step_count.sub_(1)
            raise


class DecodeBlock:
    """A block whose experts are in 4 bits, for decode steps of up to ``T`` tokens.

    ``act8`` (bf16 blocks): the experts read the norm's 8-bit output; the router always reads the full one.  Of ``params`` the
    block keeps gamma, Wg and the bias: W1, W3 and W2 may be freed once they are quantised."""

    def __init__(self, params: dict, T: int, k: int, group: int = 128, act8: bool = True, eps: float = 1e-6,
                 gate: str = "softmax", renorm: bool = False):
        W1 = params["W1"]
        E, h, f = W1.shape
        dt, dev = W1.dtype, W1.device
        self.T, self.E, self.h, self.f, self.k, self.group, self.eps = T, E, h, f, k, group, eps
        self.params = {name: params.get(name) for name in ("gamma", "Wg", "bias")}
        self.gate, self.renorm, self.dtype = gate, renorm, dt
        # a router over fewer tokens may split its sums further and need more
        route = max(B.workspace_size(B.MOE_OP_ROUTE, n, h, E, k, f, dt) for n in range(T + 1))
        self.ws = torch.zeros(max(route, B.workspace_size(B.MOE_OP_EXPERT_FFN_W4, T, h, E, k, f, dt)), dtype=torch.uint8, device=dev)
        self.w4 = []
        for name in ("W1", "W3", "W2"):
            _, K, N = params[name].shape
            q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=dev)
            scale = torch.empty(E, N, -(-K // group), dtype=torch.bfloat16, device=dev)
            B.moe_quantize_w4(params[name], group, q, scale, self.ws)
            self.w4 += [q, scale]
        d = dict(device=dev)
        self.s, self.n, self.y = (torch.empty(T, h, dtype=dt, **d) for _ in range(3))
        self.act8 = bool(act8) and dt == torch.bfloat16
        self.q = torch.empty(T, h, dtype=torch.float8_e4m3fn, **d) if self.act8 else None
        self.q_scale = torch.empty(T, -(-h // 128), **d) if self.act8 else None
        self.logits, self.probs = torch.empty(T, E, **d), torch.empty(T, E, **d)
        self.topk_idx, self.topk_w = torch.empty(T, k, dtype=torch.int32, **d), torch.empty(T, k, **d)

    def step(self, x: torch.Tensor, residual: torch.Tensor):
        """(y, s) of a batch of at most the block's T tokens: rows of the block's own buffers, which the next step overwrites."""
        p, n = self.params, x.shape[0]
        if n > self.T:
            raise ValueError(f"a batch of {n} tokens for a block of {self.T}")
        own = (self.s, self.n, self.y, self.q, self.q_scale, self.logits, self.probs, self.topk_idx, self.topk_w)
        if n != self.T:
            own = [t if t is None else t[:n] for t in own]
        s, normed, y, q, q_scale, logits, probs, topk_idx, topk_w = own
        B.moe_add_rmsnorm(x, residual, p["gamma"], self.eps, s, normed, q, q_scale, None, self.ws)
        B.moe_route(normed, p["Wg"], p["bias"], self.k, logits, probs, topk_idx, topk_w, self.ws, gate=self.gate, renorm=self.renorm)
        B.moe_expert_ffn_w4(q if self.act8 else normed, q_scale, topk_idx, topk_w, *self.w4, self.group, y, self.ws)
        return y, s
