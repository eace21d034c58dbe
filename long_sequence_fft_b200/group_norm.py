"""Group normalisation, channels last, with an activation or an activated gate
(fftconv_group_norm), differentiable.

    n = (x - mean) / sqrt(var + eps) * weight + bias,   y = act(n)  or  n * act(gate)
"""
from __future__ import annotations

from . import BF16, F16, F32, _check, _lib
from . import _ptr as _p
from .linear_attention import _no_tangents, _on, _written

ACTIVATIONS = {"none": 0, "silu": 1, "sigmoid": 2}
_CODES = None


def _code(dtype):
    """The library's code of a torch dtype; None: not one of its types."""
    global _CODES
    if _CODES is None:
        import torch
        _CODES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    return _CODES.get(dtype)


def _ld(t, C):
    """The row stride of t as rows of C channels one stride apart; None where
    it does not lie so, or where the kernels cannot read it as it lies."""
    if t.is_contiguous():
        return C if t.data_ptr() % 16 == 0 else None
    if not t.numel():
        return C
    try:
        rows = t.view(-1, C)
    except RuntimeError:
        return None
    if t.data_ptr() % 16 or (C > 1 and t.stride(-1) != 1):
        return None
    if rows.shape[0] == 1:
        return C
    return rows.stride(0) if rows.stride(0) >= C else None


def _forward(x, ld, gate, ld_gate, weight, bias, N, S, C, G, act, eps, out, keep, stream):
    import torch
    device = x.device
    with _on(device, stream) as handle:
        y = torch.empty(x.shape, dtype=x.dtype, device=device) if out is None else out
        # mean and rstd, one after the other
        stats = torch.empty((2, N, G), dtype=torch.float32, device=device) if keep else None
        mean = stats.data_ptr() if keep else None
        n = int(_lib.fftconv_group_norm_workspace_bytes(N, S, C, G, 0))
        ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
        code = _code(x.dtype)
        _check(_lib.fftconv_group_norm(_p(x), _p(gate), _p(weight), _p(bias), _p(y), mean,
                                       mean + 4 * N * G if keep else None, N, S, C, G, ld, ld_gate, code,
                                       code if weight is None else _code(weight.dtype), act, eps, _p(ws), n, handle))
    if out is not None:
        _written(out)
    return y, stats


_AUTOGRAD_FN = None


def _autograd_function():
    global _AUTOGRAD_FN
    if _AUTOGRAD_FN is not None:
        return _AUTOGRAD_FN
    import torch

    class GroupNormFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gate, weight, bias, args):
            # (one argument for all that is no tensor: autograd looks at each)
            ld, ld_gate, N, S, C, G, act, eps = args
            y, stats = _forward(x, ld, gate, ld_gate, weight, bias, N, S, C, G, act, eps, None, True, None)
            ctx.save_for_backward(x, gate, weight, bias, stats)
            ctx.args = args
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, gate, weight, bias, stats = ctx.saved_tensors
            ld, ld_gate, N, S, C, G, act, _ = ctx.args
            need = ctx.needs_input_grad
            ld_dy = _ld(dy, C)
            if ld_dy is None:
                # a gradient comes in whatever layout, and at whatever address,
                # autograd has (a copy: contiguous() would return a contiguous
                # one that is not aligned as it is)
                dy, ld_dy = dy.clone(memory_format=torch.contiguous_format), C
            device = x.device
            with _on(device, None) as handle:
                dx = torch.empty(x.shape, dtype=x.dtype, device=device)
                dgate = None if gate is None else torch.empty(x.shape, dtype=x.dtype, device=device)
                sums = None
                if weight is not None and (need[2] or need[3]):
                    sums = torch.empty((2, C), dtype=torch.float32, device=device)
                n = int(_lib.fftconv_group_norm_workspace_bytes(N, S, C, G, 1))
                ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
                code, mean = _code(x.dtype), stats.data_ptr()
                dw = None if sums is None else sums.data_ptr()
                _check(_lib.fftconv_group_norm_backward(
                    _p(x), _p(gate), _p(weight), _p(bias), _p(dy), mean, mean + 4 * N * G, _p(dx), _p(dgate), dw,
                    None if dw is None else dw + 4 * C, N, S, C, G, ld, ld_gate, ld_dy, code,
                    code if weight is None else _code(weight.dtype), act, _p(ws), n, handle))
            dweight, dbias = (None, None) if sums is None else sums.to(weight.dtype).unbind(0)
            return (dx if need[0] else None, dgate if need[1] else None, dweight if need[2] else None,
                    dbias if need[3] else None, None)

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
    weight and bias (not in forward mode, and not together with `out` or
    `stream`).  When a backward
    pass is captured into a CUDA graph, let the forward call of the same leaves
    be captured with it."""
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
    ld, ld_gate = _ld(x, C), 0 if gate is None else _ld(gate, C)
    if ld is None or ld_gate is None:
        raise ValueError(f"{'x' if ld is None else 'gate'} must be rows of contiguous channels, one stride apart, "
                         "16-byte aligned")
    _no_tangents(x, gate, weight, bias)
    grad = torch.is_grad_enabled() and (
        x.requires_grad or (gate is not None and gate.requires_grad) or
        (weight is not None and (weight.requires_grad or bias.requires_grad)))
    if grad:
        if out is not None or stream is not None:
            raise NotImplementedError("group_norm: no gradients with out= or stream=")
        return _autograd_function().apply(x, gate, weight, bias, (ld, ld_gate, N, S, C, G, act, float(eps)))
    return _forward(x, ld, gate, ld_gate, weight, bias, N, S, C, G, act, float(eps), out, False, stream)[0]
