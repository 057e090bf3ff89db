"""Python binding of the C ABI in include/moe_pft.h (ctypes; argument marshalling only).

Every function takes torch CUDA tensors that the caller allocated, passes their device
pointers and the current CUDA stream to the function of the same name in libmoe_pft.so, and
raises ``MoEError`` on a non-zero status.  There is no CPU path: without the built library or
a CUDA device the first call raises.
"""

from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_pft.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_DEVICE = (
    0, -1, -2, -3, -4, -5)
MOE_F32, MOE_BF16, MOE_E4M3 = 0, 1, 2
MOE_STATUS_BAD_INDEX, MOE_STATUS_TIMEOUT, MOE_STATUS_NOT_FINITE = 1, 2, 4
MOE_ROUTE_FROM_LOGITS, MOE_ROUTE_SIGMOID, MOE_ROUTE_RENORM = 1, 2, 4
(MOE_OP_ROUTE, MOE_OP_ROUTE_BWD, MOE_OP_PFT_BUILD, MOE_OP_DISPATCH, MOE_OP_DISPATCH_BWD,
 MOE_OP_EXPERT_FFN, MOE_OP_EXPERT_FFN_BWD, MOE_OP_COMBINE, MOE_OP_COMBINE_BWD, MOE_OP_ALL, MOE_OP_GSHARD,
 MOE_OP_ADD_RMSNORM, MOE_OP_ADD_RMSNORM_BWD, MOE_OP_ADAMW, MOE_OP_EXPERT_FFN_W4) = range(15)

# C signatures: (name, restype, argtypes).  P = pointer, I = int, Z = size_t.
_P, _I, _Z, _D = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
SIGNATURES = {
    "moe_abi_version": (_I, []),
    "moe_kernel_launches": (ctypes.c_uint64, []),
    "moe_profile_events": (_I, [ctypes.POINTER(ctypes.c_void_p), _I]),
    "moe_profile_count": (ctypes.c_uint64, []),
    "moe_debug_withhold_stage": (_I, [_I, ctypes.c_ulonglong]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_status_reset": (_I, [_P, _P]),
    "moe_check_status": (_I, [_P, _P, ctypes.POINTER(ctypes.c_int)]),
    "moe_route": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_route_bwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_pft_build": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_pft_build_noalloc": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "moe_dispatch": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "moe_dispatch_bwd": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "moe_expert_ffn": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_expert_ffn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                _P, _P, _P, _P, _P, _Z, _P]),
    "moe_expert_ffn_gather": (_I, [_P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                   _P, _Z, _P]),
    "moe_expert_ffn_bwd_gather": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                       _P, _P, _P, _P, _P, _Z, _P]),
    "moe_expert_ffn_gather_supported": (_I, [_I, _I, _I]),
    "moe_expert_ffn_fused": (_I, [_P, _P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                  _P, _P, _Z, _P]),
    "moe_combine": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "moe_gshard_gate": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_gshard_dispatch": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "moe_gshard_combine": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
    "moe_combine_bwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _Z, _P]),
    "moe_add_rmsnorm": (_I, [_P, _P, _P, ctypes.c_float, _I, _I, _I, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_add_rmsnorm_bwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _Z, _P]),
    "moe_adamw_step": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _D, _D, _D, ctypes.c_uint64,
                            _P, _Z, _P]),
    "moe_quantize_w4": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _Z, _P]),
    "moe_expert_ffn_w4": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _Z, _P]),
}


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with status {code}: {msg}")
        self.code = code


_lib = None
_marshal = None  # the module that checks tensors and takes their addresses (csrc/marshal.cpp)


def lib() -> ctypes.CDLL:
    """Load libmoe_pft.so once; raise if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _checks():
    """The checking module, loaded by the first call that needs it; raise if it is not built."""
    global _marshal
    if _marshal is None:
        try:
            from . import _marshal as M
        except ImportError as e:
            raise RuntimeError(f"_marshal.so is not built for this Python and torch ({e}): run __graft_entry__.build() first") from e
        _marshal = M
    return _marshal


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


# The current stream's handle alone: building torch's Stream object costs more than the rest of a call's marshalling.  These two
# are not of torch's public interface; without them the public one is asked.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream():
    if _raw_stream is None or _raw_device is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_raw_device())


def _call(name, *args):
    rc = getattr(_lib or lib(), name)(*args)
    if rc != MOE_OK:
        raise MoEError(name, rc, (lib().moe_last_error() or b"").decode())


def workspace_size(op: int, T: int, h: int, E: int, k: int, f: int, dtype: torch.dtype) -> int:
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(lib().moe_workspace_size(op, T, h, E, k, f, code))


def new_workspace(op: int, T: int, h: int, E: int, k: int, f: int, dtype: torch.dtype, device="cuda"):
    """A zeroed uint8 workspace of moe_workspace_size bytes (status word cleared)."""
    return torch.zeros(workspace_size(op, T, h, E, k, f, dtype), dtype=torch.uint8, device=device)


class KernelTimer:
    """Per-kernel CUDA-event timing through moe_profile_events: the library records one event
    after each of its launches, on the launching stream."""

    def __init__(self, capacity: int):
        stream = torch.cuda.current_stream()
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        for e in self.events:  # materialise the underlying cudaEvent_t
            e.record(stream)
        self._handles = (ctypes.c_void_p * capacity)(*[e.cuda_event for e in self.events])
        self.capacity = capacity

    def __enter__(self):
        rc = lib().moe_profile_events(self._handles, self.capacity)
        if rc != MOE_OK:
            raise MoEError("moe_profile_events", rc, (lib().moe_last_error() or b"").decode())
        return self

    def count(self) -> int:
        return int(lib().moe_profile_count())

    def event(self, n: int):
        return self.events[n % self.capacity]

    def __exit__(self, *exc):
        lib().moe_profile_events(None, 0)
        return False


def moe_status_reset(ws):
    _call("moe_status_reset", _p(ws), _stream())


def moe_check_status(ws) -> int:
    """Synchronise the current stream and return the device status word (0 = clean)."""
    code = ctypes.c_int(0)
    rc = lib().moe_check_status(_p(ws), _stream(), ctypes.byref(code))
    if rc not in (MOE_OK, MOE_ERR_DEVICE):
        raise MoEError("moe_check_status", rc, (lib().moe_last_error() or b"").decode())
    return code.value


def moe_debug_withhold_stage(launches: int, wait_limit_ns: int = 0):
    """Test hook: the next ``launches`` tensor-core kernel launches withhold their first pipeline
    stage, so their bounded waits run out (after ``wait_limit_ns``; 0 = the default limit) and
    they report MOE_STATUS_TIMEOUT.  ``launches=0`` cancels."""
    rc = lib().moe_debug_withhold_stage(int(launches), int(wait_limit_ns))
    if rc != MOE_OK:
        raise MoEError("moe_debug_withhold_stage", rc, (lib().moe_last_error() or b"").decode())


def gate_flags(gate: str = "softmax", renorm: bool = False) -> int:
    if gate not in ("softmax", "sigmoid"):
        raise ValueError(f"unknown gate {gate!r}")
    return (MOE_ROUTE_SIGMOID if gate == "sigmoid" else 0) | (MOE_ROUTE_RENORM if renorm else 0)


def moe_route(x, Wg, bias, k, logits, probs, topk_idx, topk_w, ws, from_logits=False, dtype=None,
              gate="softmax", renorm=False):
    T, E = logits.shape
    h = x.shape[1] if x is not None else 0
    dt = _dtype_code(x) if x is not None else (MOE_BF16 if dtype == torch.bfloat16 else MOE_F32)
    flags = gate_flags(gate, renorm) | (MOE_ROUTE_FROM_LOGITS if from_logits else 0)
    _call("moe_route", _p(x), _p(Wg), _p(bias), T, h, E, k, dt, flags, _p(logits), _p(probs),
          _p(topk_idx), _p(topk_w), _p(ws), ws.numel(), _stream())


def moe_route_bwd(x, Wg, probs, topk_idx, d_topk_w, d_logits, dWg, dx_router, ws, gate="softmax",
                  renorm=False):
    T, h = x.shape
    E = Wg.shape[1]
    k = topk_idx.shape[1]
    _call("moe_route_bwd", _p(x), _p(Wg), _p(probs), _p(topk_idx), _p(d_topk_w), T, h, E, k,
          _dtype_code(x), gate_flags(gate, renorm), _p(d_logits), _p(dWg), _p(dx_router), _p(ws),
          ws.numel(), _stream())


def moe_pft_build(topk_idx, E, num_ids, offsets, token_ids, expert_ids, slot_of, ws):
    T, k = topk_idx.shape
    _call("moe_pft_build", _p(topk_idx), T, E, k, _p(num_ids), _p(offsets), _p(token_ids),
          _p(expert_ids), _p(slot_of), _p(ws), ws.numel(), _stream())


def moe_pft_build_noalloc(topk_idx, E, num_ids, offsets, token_ids, expert_ids, slot_of):
    """moe_pft_build without a workspace: its scratch is the library's static device array,
    for callers that cannot allocate.  Calls that overlap on the GPU race."""
    T, k = topk_idx.shape
    _call("moe_pft_build_noalloc", _p(topk_idx), T, E, k, _p(num_ids), _p(offsets), _p(token_ids),
          _p(expert_ids), _p(slot_of), _stream())


def moe_dispatch(x, token_ids, k, xbuf, ws):
    T, h = x.shape
    _call("moe_dispatch", _p(x), _p(token_ids), T, k, h, _dtype_code(x), _p(xbuf), _p(ws),
          ws.numel(), _stream())


def moe_dispatch_bwd(dxbuf, slot_of, dx_add, k, dx, ws):
    T, h = dx.shape
    _call("moe_dispatch_bwd", _p(dxbuf), _p(slot_of), _p(dx_add), T, k, h, _dtype_code(dx), _p(dx),
          _p(ws), ws.numel(), _stream())


def moe_expert_ffn(xbuf, offsets, W1, W3, W2, ybuf, h1, h3, a, ws):
    Tk, h = xbuf.shape
    E, _, f = W1.shape
    _call("moe_expert_ffn", _p(xbuf), _p(offsets), _p(W1), _p(W3), _p(W2), Tk, E, h, f,
          _dtype_code(xbuf), _p(ybuf), _p(h1), _p(h3), _p(a), _p(ws), ws.numel(), _stream())


def moe_expert_ffn_bwd(dybuf, xbuf, h1, h3, a, offsets, W1, W3, W2, dxbuf, dW1, dW3, dW2, ws):
    Tk, h = xbuf.shape
    E, _, f = W1.shape
    _call("moe_expert_ffn_bwd", _p(dybuf), _p(xbuf), _p(h1), _p(h3), _p(a), _p(offsets), _p(W1),
          _p(W3), _p(W2), Tk, E, h, f, _dtype_code(xbuf), _p(dxbuf), _p(dW1), _p(dW3), _p(dW2),
          _p(ws), ws.numel(), _stream())


def moe_expert_ffn_gather(x, token_ids, offsets, W1, W3, W2, ybuf, h1, h3, a, ws):
    T, h = x.shape
    Tk = token_ids.shape[0]
    E, _, f = W1.shape
    _call("moe_expert_ffn_gather", _p(x), _p(token_ids), T, _p(offsets), _p(W1), _p(W3), _p(W2), Tk, E,
          h, f, _dtype_code(x), _p(ybuf), _p(h1), _p(h3), _p(a), _p(ws), ws.numel(), _stream())


def moe_expert_ffn_bwd_gather(dybuf, x, token_ids, h1, h3, a, offsets, W1, W3, W2, dxbuf, dW1, dW3, dW2,
                              ws):
    T, h = x.shape
    Tk = token_ids.shape[0]
    E, _, f = W1.shape
    _call("moe_expert_ffn_bwd_gather", _p(dybuf), _p(x), _p(token_ids), T, _p(h1), _p(h3), _p(a),
          _p(offsets), _p(W1), _p(W3), _p(W2), Tk, E, h, f, _dtype_code(x), _p(dxbuf), _p(dW1), _p(dW3),
          _p(dW2), _p(ws), ws.numel(), _stream())


def moe_expert_ffn_gather_supported(h: int, f: int, dtype: torch.dtype) -> bool:
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return bool(lib().moe_expert_ffn_gather_supported(h, f, code))


def moe_expert_ffn_fused(xbuf, x, token_ids, slot_of, topk_w, offsets, W1, W3, W2, ybuf, h1, h3, a, y, ws):
    """Expert FFN with the dispatch (xbuf None: rows gathered from x) and/or the combine (y not
    None) folded into its GEMMs."""
    T, k = topk_w.shape
    Tk = token_ids.shape[0]
    E, h, f = W1.shape
    dt = (xbuf if xbuf is not None else x).dtype
    code = MOE_BF16 if dt == torch.bfloat16 else MOE_F32
    _call("moe_expert_ffn_fused", _p(xbuf), _p(x), _p(token_ids), T, k, _p(slot_of), _p(topk_w), _p(offsets),
          _p(W1), _p(W3), _p(W2), Tk, E, h, f, code, _p(ybuf), _p(h1), _p(h3), _p(a), _p(y), _p(ws), ws.numel(),
          _stream())


def moe_combine(ybuf, slot_of, topk_w, y, ws):
    T, h = y.shape
    k = topk_w.shape[1]
    _call("moe_combine", _p(ybuf), _p(slot_of), _p(topk_w), T, k, h, _dtype_code(y), _p(y), _p(ws),
          ws.numel(), _stream())


def moe_combine_bwd(dy, ybuf, slot_of, topk_w, dybuf, d_topk_w, ws):
    T, h = dy.shape
    k = topk_w.shape[1]
    _call("moe_combine_bwd", _p(dy), _p(ybuf), _p(slot_of), _p(topk_w), T, k, h, _dtype_code(dy),
          _p(dybuf), _p(d_topk_w), _p(ws), ws.numel(), _stream())


def moe_gshard_gate(topk_idx, topk_w, E, C, dispatch_mask, combine_w, loads, ws):
    """Capacity-buffer gate: dispatch_mask [T,E,C] (activation dtype) and combine_w [T,E,C] fp32."""
    T, k = topk_idx.shape
    _call("moe_gshard_gate", _p(topk_idx), _p(topk_w), T, E, k, C, _dtype_code(dispatch_mask),
          _p(dispatch_mask), _p(combine_w), _p(loads), _p(ws), ws.numel(), _stream())


def moe_gshard_dispatch(x, dispatch_mask, xe, ws):
    """xe [E,C,h] = the contraction of dispatch_mask [T,E,C] with x [T,h] over the tokens."""
    T, E, C = dispatch_mask.shape
    h = x.shape[1]
    _call("moe_gshard_dispatch", _p(x), _p(dispatch_mask), T, E, C, h, _dtype_code(x), _p(xe), _p(ws),
          ws.numel(), _stream())


def moe_gshard_combine(combine_w, ye, y, ws):
    """y [T,h] = the contraction of combine_w [T,E,C] with ye [E,C,h] over (e, c)."""
    T, E, C = combine_w.shape
    h = ye.shape[2]
    _call("moe_gshard_combine", _p(combine_w), _p(ye), T, E, C, h, _dtype_code(ye), _p(y), _p(ws), ws.numel(),
          _stream())


def _check(t, name, dtype, shape):
    """Refuse a tensor whose type, shape or place the call would misread (None passes); returns its address."""
    return (_marshal or _checks()).pointer(t, name, dtype, shape)


def moe_add_rmsnorm(x, residual, gamma, eps, s, y, q, q_scale, rstd, ws):
    """s = x + residual (both None: s is x) and its RMSNorm: y in x's dtype and/or q (float8_e4m3fn) with
    q_scale [T, ceil(h/128)] fp32; rstd [T] fp32 (or None) is what the backward needs."""
    shape, dt = x.shape, x.dtype
    T, h = shape
    _call("moe_add_rmsnorm", _check(x, "x", dt, shape), _check(residual, "residual", dt, shape), _check(gamma, "gamma", torch.float32, (h,)),
          eps, T, h, _dtype_code(x), _check(s, "s", dt, shape), _check(y, "y", dt, shape),
          _check(q, "q", torch.float8_e4m3fn, shape), _check(q_scale, "q_scale", torch.float32, (T, (h + 127) // 128)),
          _check(rstd, "rstd", torch.float32, (T,)), _p(ws), ws.numel(), _stream())


def moe_add_rmsnorm_bwd(dy, s, gamma, rstd, ds_add, ds, dgamma, ws):
    """ds = ds_add (or 0) + the norm's gradient for dy; dgamma [h] fp32."""
    shape, dt = s.shape, s.dtype
    T, h = shape
    _call("moe_add_rmsnorm_bwd", _check(dy, "dy", dt, shape), _check(s, "s", dt, shape), _check(gamma, "gamma", torch.float32, (h,)),
          _check(rstd, "rstd", torch.float32, (T,)), _check(ds_add, "ds_add", dt, shape), T, h, _dtype_code(s),
          _check(ds, "ds", dt, shape), _check(dgamma, "dgamma", torch.float32, (h,)), _p(ws), ws.numel(), _stream())


def moe_adamw_step(params, grads, masters, m, v, m_scale, v_scale, weight_decay, lr, step, grad_scale, beta1, beta2,
                   eps, seed, ws):
    """One AdamW step over lists of tensors, in place.  bf16 parameters have an fp32 master (None for fp32 ones;
    ``masters`` may be None when there are none).  States: fp32, or with ``m_scale`` and ``v_scale`` (lists of fp32, one
    value per 256 elements) float8_e4m3fn m and float8_e5m2 v.  ``weight_decay``: a number, or one per tensor.  ``lr``
    (fp32[1]), ``step`` (int32[1], this step's number) and ``grad_scale`` (fp32[1] or None) are on the device."""
    n = len(params)
    p, g, masters, m, v, m_scale, v_scale, sizes, codes = (_marshal or _checks()).optimizer(params, grads, masters, m, v, m_scale, v_scale)
    if not isinstance(weight_decay, (list, tuple)):
        weight_decay = [weight_decay] * n
    elif len(weight_decay) != n:
        raise ValueError(f"weight_decay: {len(weight_decay)} numbers for {n} parameters")
    wd = (ctypes.c_float * n)(*weight_decay)
    _call("moe_adamw_step", n, p, g, masters, m, v, m_scale, v_scale, sizes, wd, codes, 32 if m_scale is None else 8,
          _check(lr, "lr", torch.float32, (1,)), _check(step, "step", torch.int32, (1,)),
          _check(grad_scale, "grad_scale", torch.float32, (1,)), beta1, beta2, eps, seed, _p(ws), ws.numel(), _stream())


def moe_quantize_w4(W, group, q, scale, ws):
    """W [E, K, N] to 4 bits: q [E, N, K/2] uint8 (two inputs a byte) and scale [E, N, ceil(K/group)] bf16."""
    E, K, N = W.shape
    _call("moe_quantize_w4", _p(W), E, K, N, _dtype_code(W), group, _check(q, "q", torch.uint8, (E, N, K // 2)),
          _check(scale, "scale", torch.bfloat16, (E, N, -(-K // group))), _p(ws), ws.numel(), _stream())


def moe_expert_ffn_w4(x, x_scale, topk_idx, topk_w, W1q, W1s, W3q, W3s, W2q, W2s, group, y, ws):
    """The routed experts of a few tokens over 4-bit weights (moe_quantize_w4 of W1, W3 and W2): y [T, h] from x (y's
    dtype, or float8_e4m3fn with x_scale [T, ceil(h/128)]) and the gate's topk_idx and topk_w [T, k]."""
    T, k = topk_idx.shape
    h = y.shape[1]
    E, f, _ = W1q.shape
    dt, u8, bf = y.dtype, torch.uint8, torch.bfloat16
    q8 = x.dtype == torch.float8_e4m3fn
    up, down = (E, f, -(-h // group)), (E, h, -(-f // group))
    _call("moe_expert_ffn_w4", _check(x, "x", x.dtype if q8 else dt, (T, h)),
          _check(x_scale, "x_scale", torch.float32, (T, -(-h // 128))), _check(topk_idx, "topk_idx", torch.int32, (T, k)),
          _check(topk_w, "topk_w", torch.float32, (T, k)), _check(W1q, "W1q", u8, (E, f, h // 2)), _check(W1s, "W1s", bf, up),
          _check(W3q, "W3q", u8, (E, f, h // 2)), _check(W3s, "W3s", bf, up), _check(W2q, "W2q", u8, (E, h, f // 2)),
          _check(W2s, "W2s", bf, down), T, k, E, h, f, group, MOE_E4M3 if q8 else _dtype_code(y), _dtype_code(y),
          _check(y, "y", dt, (T, h)), _p(ws), ws.numel(), _stream())
