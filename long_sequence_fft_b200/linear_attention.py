"""Causal linear attention with a decay for each head: the prompt form
(fftconv_linear_attention, differentiable) and the single-token form
(fftconv_linear_attention_step).

    S_t = g S_{t-1} + k_t v_t^T,    o_t = scale * q_t S_t,    g = exp(log_decay[h])
"""
from __future__ import annotations

import ctypes
import struct

from . import BF16, F16, _check, _i64, _lib, _vp
from . import _ptr as _p

_CODES = None
_Pair = _i64 * 2


class _Shape(ctypes.Structure):
    _fields_ = [("B", _i64), ("T", _i64), ("nseq", _i64), ("H", _i64), ("Hq", _i64), ("Hk", _i64), ("Hv", _i64),
                ("K", _i64), ("V", _i64), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("zero_rest", ctypes.c_int32), ("q_stride", _i64 * 3), ("k_stride", _i64 * 3),
                ("v_stride", _i64 * 3), ("o_stride", _i64 * 3)]


# its bytes: quicker to write than the fields of a ctypes structure
_pack_shape = struct.Struct("=9qifi4x12q")
assert _pack_shape.size == ctypes.sizeof(_Shape)


def _dtype_of(t, name):
    global _CODES
    if _CODES is None:
        import torch
        _CODES = {torch.float16: F16, torch.bfloat16: BF16}
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} has dtype {t.dtype}; linear attention takes float16 or bfloat16")
    return code


class _On:
    """Make `device` and `stream` (None: the device's current one; a
    torch.cuda.Stream or a raw handle) current, so that what is allocated
    inside belongs to the stream that uses it; enters with the raw handle.
    Nothing is switched, or asked of torch's slower interfaces, for a call on
    the current device and stream: small calls are all overhead."""
    __slots__ = ("device", "stream", "outer")

    def __init__(self, device, stream):
        self.device, self.stream, self.outer = device, stream, ()

    def __enter__(self):
        import torch
        stream = self.stream
        if stream is None and torch._C._cuda_getDevice() == self.device.index:
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        device = torch.cuda.device(self.device)
        device.__enter__()
        self.outer = (device,)
        if stream is None:
            return torch.cuda.current_stream().cuda_stream
        if isinstance(stream, int):
            # 0 is the legacy default stream, which has no external handle
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        inside = torch.cuda.stream(stream)
        inside.__enter__()
        self.outer = (inside, device)
        return stream.cuda_stream

    def __exit__(self, *exc):
        for o in self.outer:
            o.__exit__(*exc)
        return False


_on = _On


def _written(t):
    """Mark the caller's tensor as written in place, which a launch through its
    address does not: a backward pass that saved it then raises, as for torch's
    own in-place operations."""
    import torch
    torch.autograd.graph.increment_version(t)


def _no_tangents(*tensors):
    """Refuse dual tensors: they do not require a gradient, so a call would
    return a result without a tangent, which stands for a derivative of zero."""
    import torch
    ad = torch.autograd.forward_ad
    if getattr(ad, "_current_level", 0) >= 0:                 # (inside a dual_level)
        for t in tensors:
            if t is not None and ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError("linear attention and group norm have no forward-mode derivatives")


def _need(t, name, dtype, shape, device):
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _need_contiguous(t, name, dtype, shape, device):
    _need(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_heads(log_decay, device, *heads):
    import torch
    if log_decay.dim() != 1 or log_decay.shape[0] == 0:
        raise ValueError("log_decay must be a vector of one value for each head")
    H = log_decay.shape[0]
    _need_contiguous(log_decay, "log_decay", torch.float32, (H,), device)
    if log_decay.requires_grad and torch.is_grad_enabled():
        raise NotImplementedError("linear attention has no gradient for log_decay: detach it")
    for name, h in zip("qkv", heads):
        if h < 1 or H % h:
            raise ValueError(f"{name} has {h} heads, which do not divide the {H} heads of log_decay")
    return H


def _check_readable(*tensors):
    for t, name in zip(tensors, "qkv"):
        if not ((t.is_contiguous() and t.data_ptr() % 16 == 0) or not t.numel() or _usable(t)):
            raise ValueError(f"{name}: the last index must be contiguous, and the other strides and the data's "
                             "address multiples of 16 bytes (not expanded)")


def _shape_of(q, k, v, o_shape_stride, log_decay, nseq, scale, zero_rest):
    (B, T, Hq, K), Hk, (Hv, V) = q.shape, k.shape[2], v.shape[2:]
    return _pack_shape.pack(B, T, nseq, log_decay.shape[0], Hq, Hk, Hv, K, V, _dtype_of(q, "q"), scale, zero_rest,
                            *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *o_shape_stride[:3])


def _workspace(shape, backward, device):
    import torch
    n = int(_lib.fftconv_linear_attention_workspace_bytes(shape, backward))
    return (torch.empty(n, dtype=torch.uint8, device=device) if n else None), n


def _forward(q, k, v, log_decay, initial, cu, scale, want_state, out, stream):
    import torch
    B, T = q.shape[:2]
    H, K, V = log_decay.shape[0], q.shape[3], v.shape[3]
    nseq = 0 if cu is None else cu.shape[0] - 1
    given = out
    with _on(q.device, stream) as handle:
        zero_rest = out is None
        if out is None:
            out = torch.empty((B, T, H, V), dtype=q.dtype, device=q.device)
        shape = _shape_of(q, k, v, out.stride(), log_decay, nseq, scale, zero_rest)
        state = None
        if want_state:
            state = torch.empty((nseq if cu is not None else B, H, K, V), dtype=torch.float32, device=q.device)
        ws, n = _workspace(shape, 0, q.device)
        _check(_lib.fftconv_linear_attention(shape, _p(q), _p(k), _p(v), _p(log_decay), _p(initial),
                                             _p(cu), _p(out), _p(state), _p(ws), n, handle))
    if given is not None:
        _written(given)
    return out, state


def _backward(q, k, v, log_decay, initial, cu, scale, do, dstate, want_initial):
    import torch
    nseq = 0 if cu is None else cu.shape[0] - 1
    with _on(q.device, None) as handle:
        shape = _shape_of(q, k, v, do.stride(), log_decay, nseq, scale, 1)
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        dinitial = torch.empty_like(initial) if want_initial else None
        ws, n = _workspace(shape, 1, q.device)
        _check(_lib.fftconv_linear_attention_backward(shape, _p(q), _p(k), _p(v), _p(log_decay),
                                                      _p(initial), _p(cu), _p(do), _p(dstate), _p(dq), _p(dk), _p(dv),
                                                      _p(dinitial), _p(ws), n, handle))
    return dq, dk, dv, dinitial


def _usable(t):
    """Whether a kernel can read t as it lies (last index contiguous, 16-byte
    aligned rows)."""
    return t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(
        n == 1 or (s > 0 and s % 8 == 0) for n, s in zip(t.shape[:-1], t.stride()[:-1]))


_AUTOGRAD_FN = None


def _autograd_function():
    global _AUTOGRAD_FN
    if _AUTOGRAD_FN is not None:
        return _AUTOGRAD_FN
    import torch

    class LinearAttentionFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, initial, log_decay, cu, scale, want_state):
            out, state = _forward(q, k, v, log_decay, initial, cu, scale, want_state, None, None)
            ctx.save_for_backward(q, k, v, initial, log_decay, cu)
            ctx.scale = scale
            ctx.set_materialize_grads(False)
            return out, state

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, do, dstate):
            q, k, v, initial, log_decay, cu = ctx.saved_tensors
            if do is None and dstate is None:
                return (None,) * 8
            if do is None:
                do = torch.zeros(q.shape[:2] + (log_decay.shape[0], v.shape[3]), dtype=q.dtype, device=q.device)
            # a gradient comes in whatever layout autograd has: an expanded
            # scalar, a transposed view, a piece of a concatenation's gradient
            # at any address (a copy, then: contiguous() would return it as it is)
            if not _usable(do):
                do = do.clone(memory_format=torch.contiguous_format)
            if dstate is not None and not (dstate.is_contiguous() and dstate.data_ptr() % 16 == 0):
                dstate = dstate.clone(memory_format=torch.contiguous_format)
            need = ctx.needs_input_grad
            dq, dk, dv, dinitial = _backward(q, k, v, log_decay, initial, cu, ctx.scale, do, dstate,
                                             initial is not None and need[3])
            return (dq if need[0] else None, dk if need[1] else None, dv if need[2] else None, dinitial, None, None,
                    None, None)

    _AUTOGRAD_FN = LinearAttentionFunction
    return _AUTOGRAD_FN


def linear_attention(q, k, v, log_decay, *, scale=None, initial_state=None, cu_seqlens=None, return_state=False,
                     out=None, stream=None):
    """Causal linear attention over whole sequences (include/fftconv.h).

    q [B, T, Hq, K], k [B, T, Hk, K], v [B, T, Hv, V], fp16 or bf16, last index
    contiguous, other strides multiples of 8 elements; log_decay [H] fp32, on
    the device; Hq, Hk and Hv divide H (head h reads head h // (H // Hq)).
    K and V: multiples of 8 up to 128.  scale: K ** -0.5 unless given.
    cu_seqlens (int32 on the device, [n + 1] offsets; B = 1): n packed
    sequences of any lengths; rows outside them are zero (with `out`: left as
    they were), and so are their gradients.
    initial_state [B or n, H, K, V] fp32: the states before the first tokens.

    Returns o [B, T, H, V], or (o, state) with return_state: state is what
    linear_attention_step and a later call's initial_state take.  (o of calls
    with and without return_state, or with other tokens beside a sequence's,
    can differ in its last bits: include/fftconv.h.)  The results are complete
    unless linear_attention_status() reports a wait that gave up.
    Differentiable in q, k, v and initial_state (not in log_decay, not in
    forward mode, and not together with `out` or `stream`).  When a backward pass is captured into a
    CUDA graph, let the forward call of the same leaves be captured with it."""
    import torch
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must have 4 dimensions: batch, token, head, channel")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    B, T, Hq, K = q.shape
    V = v.shape[3]
    device = q.device
    _dtype_of(q, "q")
    _need(k, "k", q.dtype, (B, T, k.shape[2], K), device)
    _need(v, "v", q.dtype, (B, T, v.shape[2], V), device)
    _check_readable(q, k, v)
    H = _check_heads(log_decay, device, Hq, k.shape[2], v.shape[2])
    n = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("packed sequences (cu_seqlens) need a batch of 1")
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must be a vector of at least two offsets")
        n = cu_seqlens.shape[0] - 1
        _need_contiguous(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), device)
    if initial_state is not None:
        _need_contiguous(initial_state, "initial_state", torch.float32, (n, H, K, V), device)
    _no_tangents(q, k, v, log_decay, initial_state)
    scale = K ** -0.5 if scale is None else float(scale)
    grad = torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or
                                        (initial_state is not None and initial_state.requires_grad))
    if grad:
        if out is not None or stream is not None:
            raise NotImplementedError("linear_attention: no gradients with out= or stream=")
        o, state = _autograd_function().apply(q, k, v, initial_state, log_decay, cu_seqlens, scale, return_state)
        return (o, state) if return_state else o
    if out is not None:
        _need(out, "out", q.dtype, (B, T, H, V), device)
        if out.numel() and not _usable(out):
            raise ValueError("out: the last index must be contiguous, and the other strides and the data's address "
                             "multiples of 16 bytes")
    o, state = _forward(q, k, v, log_decay, initial_state, cu_seqlens, scale, return_state, out, stream)
    return (o, state) if return_state else o


def linear_attention_step(q, k, v, log_decay, state, *, slots=None, scale=None, out=None, stream=None):
    """One token of B sequences: state <- g state + k v^T in place, returns
    o [B, H, V] = scale * q state.

    q [B, Hq, K], k [B, Hk, K], v [B, Hv, V], fp16 or bf16, last index
    contiguous; state [pool, H, K, V] fp32, contiguous.  slots (int32 on the
    device, [B]): the state of each row; a row whose slot is outside the pool,
    or that an earlier row names already, is idle (zero output, no state
    touched).  Without slots row b uses state b.  No gradients; state and out
    count as written in place for gradients of other calls that saved them."""
    import torch
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must have 3 dimensions: batch, head, channel")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    B, Hq, K = q.shape
    V = v.shape[2]
    device = q.device
    code = _dtype_of(q, "q")
    _need(k, "k", q.dtype, (B, k.shape[1], K), device)
    _need(v, "v", q.dtype, (B, v.shape[1], V), device)
    _check_readable(q, k, v)
    H = _check_heads(log_decay, device, Hq, k.shape[1], v.shape[1])
    if state.dim() != 4:
        raise ValueError("state must have 4 dimensions: sequence, head, K, V")
    pool = state.shape[0]
    _need_contiguous(state, "state", torch.float32, (B if slots is None else pool, H, K, V), device)
    if slots is not None:
        _need_contiguous(slots, "slots", torch.int32, (B,), device)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or state.requires_grad):
        raise NotImplementedError("linear_attention_step has no gradients: use linear_attention, or torch.no_grad()")
    _no_tangents(q, k, v, log_decay, state)
    scale = K ** -0.5 if scale is None else float(scale)
    given = out
    with _on(device, stream) as handle:
        if out is None:
            out = torch.empty((B, H, V), dtype=q.dtype, device=device)
        else:
            _need_contiguous(out, "out", q.dtype, (B, H, V), device)
        _check(_lib.fftconv_linear_attention_step(
            _p(q), _p(k), _p(v), _p(log_decay), _p(state), _p(slots), _p(out), B, pool, H, Hq, k.shape[1],
            v.shape[1], K, V, code, scale, _Pair(*q.stride()[:2]), _Pair(*k.stride()[:2]), _Pair(*v.stride()[:2]),
            handle))
    _written(state)
    if given is not None:
        _written(given)
    return out


def linear_attention_status(stream=None) -> int:
    """Synchronise the stream and return (and reset) the status of the linear
    attention kernels on the current device: 0, or ERR_TIMEOUT once a bounded
    device-side wait gave up."""
    import torch
    handle = torch.cuda.current_stream().cuda_stream if stream is None else \
        stream if isinstance(stream, int) else stream.cuda_stream
    return int(_lib.fftconv_linear_attention_status(_vp(handle)))
