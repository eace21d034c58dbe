"""Group normalisation, channels last, with an activation or an activated gate
(fftconv_group_norm), differentiable.

    n = (x - mean) / sqrt(var + eps) * weight + bias,   y = act(n)  or  n * act(gate)
"""
from __future__ import annotations

from . import BF16, F16, F32, _check, _lib
from . import _ptr as _p
from .linear_attention import _on

ACTIVATIONS = {"none": 0, "silu": 1, "sigmoid": 2}
_CODES = None


def _code(dtype):
    """The library's code of a torch dtype; None: not one of its types."""
    global _CODES
    if _CODES is None:
        import torch
        _CODES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    return _CODES.get(dtype)


def _rows(t, C):
    """t as rows of C channels one stride apart (None: it does not lie so), and
    whether the kernels can read it as it lies."""
    if t.stride(-1) != 1 and C > 1:
        return None
    try:
        return t.view(-1, C)
    except RuntimeError:
        return None


def _checked_rows(t, C, name):
    r = _rows(t, C)
    if t.numel() and (r is None or (r.shape[0] > 1 and r.stride(0) < C) or t.data_ptr() % 16):
        raise ValueError(f"{name} must be rows of contiguous channels, one stride apart, 16-byte aligned")
    return t.reshape(-1, C) if r is None else r


def _ld(r, C):
    return r.stride(0) if r.shape[0] > 1 else C


def _forward(x2, gate2, weight, bias, N, S, C, G, act, eps, out, keep, stream, shape):
    import torch
    with _on(x2.device, stream) as handle:
        y = torch.empty(shape, dtype=x2.dtype, device=x2.device) if out is None else out
        mean = rstd = None
        if keep:
            mean, rstd = torch.empty((2, N, G), dtype=torch.float32, device=x2.device).unbind(0)
        n = int(_lib.fftconv_group_norm_workspace_bytes(N, S, C, G, 0))
        ws = torch.empty(n, dtype=torch.uint8, device=x2.device) if n else None
        _check(_lib.fftconv_group_norm(_p(x2), _p(gate2), _p(weight), _p(bias), _p(y), _p(mean), _p(rstd), N, S, C, G,
                                       _ld(x2, C), 0 if gate2 is None else _ld(gate2, C), _code(x2.dtype),
                                       _code(x2.dtype if weight is None else weight.dtype), act, eps, _p(ws), n,
                                       handle))
    return y, mean, rstd


_AUTOGRAD_FN = None


def _autograd_function():
    global _AUTOGRAD_FN
    if _AUTOGRAD_FN is not None:
        return _AUTOGRAD_FN
    import torch

    class GroupNormFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gate, weight, bias, N, S, C, G, act, eps):
            y, mean, rstd = _forward(_rows(x, C), None if gate is None else _rows(gate, C), weight, bias, N, S, C, G,
                                     act, eps, None, True, None, x.shape)
            ctx.save_for_backward(x, gate, weight, bias, mean, rstd)
            ctx.args = (N, S, C, G, act)
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, gate, weight, bias, mean, rstd = ctx.saved_tensors
            N, S, C, G, act = ctx.args
            x2, gate2, dy2 = _rows(x, C), None if gate is None else _rows(gate, C), _rows(dy, C)
            # a gradient comes in whatever layout autograd has
            if dy2 is None or dy2.data_ptr() % 16 or _ld(dy2, C) < C:
                dy2 = dy.contiguous().view(-1, C)
            need = ctx.needs_input_grad
            with _on(x.device, None) as handle:
                dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
                dgate = None if gate is None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
                dw = db = None
                if weight is not None and (need[2] or need[3]):
                    dw, db = torch.empty((2, C), dtype=torch.float32, device=x.device).unbind(0)
                n = int(_lib.fftconv_group_norm_workspace_bytes(N, S, C, G, 1))
                ws = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
                _check(_lib.fftconv_group_norm_backward(
                    _p(x2), _p(gate2), _p(weight), _p(bias), _p(dy2), _p(mean), _p(rstd), _p(dx), _p(dgate), _p(dw),
                    _p(db), N, S, C, G, _ld(x2, C), 0 if gate is None else _ld(gate2, C), _ld(dy2, C),
                    _code(x.dtype), _code(x.dtype if weight is None else weight.dtype), act, _p(ws), n,
                    handle))
            return (dx if need[0] else None, dgate if need[1] else None, dw.to(weight.dtype) if need[2] else None,
                    db.to(bias.dtype) if need[3] else None, None, None, None, None, None, None)

    _AUTOGRAD_FN = GroupNormFunction
    return _AUTOGRAD_FN


def group_norm(x, groups, weight=None, bias=None, *, gate=None, activation="none", eps=1e-5, out=None, stream=None):
    """Group normalisation of x [N, ..., C] over the positions between the
    first and the last index and the C / groups channels of each group
    (include/fftconv.h): y = act(n), or n * act(gate) with a gate of x's shape.

    x [N, C] has one position a sample: the head norm and gate behind
    linear_attention (o.view(B * T, H * V), groups = H).  fp32, fp16 or bf16;
    weight and bias [C], both or neither, in x's type or fp32.  x and gate may
    be rows of wider tensors (last index contiguous, one row stride).
    activation: "none", "silu" or "sigmoid".  Differentiable in x, gate,
    weight and bias (not together with `out` or `stream`)."""
    import torch
    if x.dim() < 2:
        raise ValueError("x must have at least 2 dimensions: sample, ..., channel")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if _code(x.dtype) is None:
        raise ValueError(f"x has dtype {x.dtype}; group norm takes float32, float16 or bfloat16")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
    N, C, G = x.shape[0], x.shape[-1], int(groups)
    if C == 0 or G < 1 or C % G:
        raise ValueError(f"groups ({groups}) must divide the {C} channels")
    S = 1
    for n in x.shape[1:-1]:
        S *= n
    if (weight is None) != (bias is None):
        raise ValueError("weight and bias: both or neither")
    if weight is not None:
        for t, name in ((weight, "weight"), (bias, "bias")):
            if t.device != x.device or t.shape != (C,) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous vector of {C} on {x.device}")
            if t.dtype != x.dtype and t.dtype != torch.float32:
                raise ValueError(f"{name} must be {x.dtype} or float32")
        if weight.dtype != bias.dtype:
            raise ValueError("weight and bias must have the same dtype")
    if gate is not None and (gate.device != x.device or gate.dtype != x.dtype or gate.shape != x.shape):
        raise ValueError("gate must have x's shape, dtype and device")
    if out is not None and (out.shape != x.shape or out.dtype != x.dtype or out.device != x.device or
                            not out.is_contiguous() or (out.numel() and out.data_ptr() % 16)):
        raise ValueError("out must be contiguous, 16-byte aligned, and have x's shape, dtype and device")
    x2 = _checked_rows(x, C, "x")
    gate2 = None if gate is None else _checked_rows(gate, C, "gate")
    grad = torch.is_grad_enabled() and (
        x.requires_grad or (gate is not None and gate.requires_grad) or
        (weight is not None and (weight.requires_grad or bias.requires_grad)))
    if grad:
        if out is not None or stream is not None:
            raise NotImplementedError("group_norm: no gradients with out= or stream=")
        return _autograd_function().apply(x, gate, weight, bias, N, S, C, G, act, float(eps))
    return _forward(x2, gate2, weight, bias, N, S, C, G, act, float(eps), out, False, stream, x.shape)[0]
