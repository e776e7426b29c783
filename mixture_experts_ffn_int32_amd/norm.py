"""Python binding of the norms around a block: ``residual_norm`` and ``rms_norm``.

Argument marshalling only; the kernels are those of csrc/norm.hip behind
hmm_residual_norm and hmm_residual_norm_backward.
"""

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .moe import _aligned, _ptr, _stream

_MAX_H = 16384
_DTYPES = {torch.bfloat16: _lib.HMM_BF16, torch.float32: _lib.HMM_F32}


def _check_tensor(name, t, device=None, dtypes=(torch.bfloat16,)):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a HIP device (got %s)" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s (got %s)" % (name, " or ".join(str(d) for d in dtypes), t.dtype))


def _check_weight(name, w, stream, H):
    _check_tensor(name, w, stream.device, tuple(_DTYPES))
    if tuple(w.shape) != (H,):
        raise ValueError("%s must be [H] with H = %d (got %s)" % (name, H, tuple(w.shape)))


def _check_stream(name, r):
    _check_tensor(name, r, None, tuple(_DTYPES))
    if r.dim() != 2 or r.shape[1] < 8 or r.shape[1] % 8 or r.shape[1] > _MAX_H:
        raise ValueError("%s must be [T,H] with H a multiple of 8 in [8, %d] (got %s)" % (name, _MAX_H, tuple(r.shape)))


def _check_scalar(name, v, positive):
    v = float(v)
    if not math.isfinite(v) or abs(v) > torch.finfo(torch.float32).max or (positive and v < torch.finfo(torch.float32).tiny):
        raise ValueError("%s must be a %s float32 (got %r)" % (name, "positive normal" if positive else "finite", v))
    return v


def _gate_kind(gate, T, H):
    """The gate's kind by its shape: (H,) per channel, (T, 1) per token, (T, H) full."""
    if gate is None:
        return _lib.HMM_GATE_NONE
    shape = tuple(gate.shape)
    if shape == (H,):
        return _lib.HMM_GATE_CHANNEL
    if shape == (T, 1):
        return _lib.HMM_GATE_TOKEN
    if shape == (T, H):
        return _lib.HMM_GATE_FULL
    raise ValueError("gate must be [H], [T,1] or [T,H] with T = %d, H = %d (got %s)" % (T, H, shape))


class ResidualNormFunction(torch.autograd.Function):
    """Forward calls hmm_residual_norm; backward calls hmm_residual_norm_backward.  y None: the norm alone."""

    @staticmethod
    def forward(ctx, y, residual, norm_weight, post_weight, gate, scale, eps):
        T, H = residual.shape
        kind = _gate_kind(gate, T, H)
        wt = norm_weight.dtype
        prob = _lib.NormProblem(T, H, _DTYPES[residual.dtype], _DTYPES[wt], kind, eps, scale)
        r, w = _aligned(residual), _aligned(norm_weight)
        y_ = None if y is None else _aligned(y)
        wp = None if post_weight is None else _aligned(post_weight)
        g = None if gate is None else _aligned(gate)
        dev = r.device
        grad = any(ctx.needs_input_grad)
        with torch.cuda.device(dev):
            out = None if y is None else torch.empty_like(r)
            normed = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
            rstd = torch.empty((2, T), dtype=torch.float32, device=dev) if grad else None
            if T > 0:
                _lib.check(_lib.load().hmm_residual_norm(ctypes.byref(prob), _ptr(y_), _ptr(r), _ptr(w), _ptr(wp), _ptr(g),
                                                         _ptr(out), _ptr(normed), _ptr(rstd), _stream(dev)))
        if grad:
            ctx.set_materialize_grads(False)
            ctx.prob = prob
            ctx.save_for_backward(y_, r if y is None else out, w, wp, g, rstd)
        return normed if y is None else (out, normed)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        d_out, d_normed = grads if len(grads) == 2 else (None, grads[0])
        y, r, w, wp, g, rstd = ctx.saved_tensors
        prob = ctx.prob
        if d_out is None and d_normed is None:
            return (None,) * 7
        dev = r.device
        d_out = None if d_out is None else _aligned(d_out, r.dtype)
        d_normed = None if d_normed is None else _aligned(d_normed, torch.bfloat16)
        with torch.cuda.device(dev):
            lib = _lib.load()
            dy = None if y is None else torch.empty_like(y)
            dr, dw = torch.empty_like(r), torch.empty_like(w)
            dwp = None if wp is None else torch.empty_like(wp)
            dg = None if g is None else torch.empty_like(g)
            if prob.T == 0:
                for t in (dw, dwp, dg):
                    if t is not None:
                        t.zero_()
            else:
                ws = ctypes.c_size_t()
                _lib.check(lib.hmm_residual_norm_backward_sizes(ctypes.byref(prob), ctypes.byref(ws)))
                work = torch.empty(ws.value, dtype=torch.uint8, device=dev)
                _lib.check(lib.hmm_residual_norm_backward(
                    ctypes.byref(prob), _ptr(d_out), _ptr(d_normed), _ptr(y), _ptr(r), _ptr(w), _ptr(wp), _ptr(g),
                    _ptr(rstd), _ptr(dy), _ptr(dr), _ptr(dw), _ptr(dwp), _ptr(dg), _ptr(work), ws.value, _stream(dev)))
        return dy, dr, dw, dwp, dg, None, None


def residual_norm(y, residual, norm_weight, *, post_weight=None, gate=None, residual_scale=1.0, eps=1e-6):
    """(residual_out, normed): the norm after a block, its gate, the residual sum and the next block's norm, fused.

    With y bf16 [T,H] the block's output and residual [T,H] (bf16 or float32) the stream before it:
    u = y / sqrt(mean(y^2) + eps) (u = y without ``post_weight``);
    residual_out = residual + residual_scale * gate * post_weight * u, rounded to the residual's type;
    normed = residual_out / sqrt(mean(residual_out^2) + eps) * norm_weight, bf16, of the stored residual_out.
    norm_weight and post_weight are [H], bf16 or float32; gate is bf16 and multiplies per channel
    ([H]), per token ([T,1]) or per element ([T,H]).  Sums are float32.  Differentiable in all five tensors.
    """
    _check_stream("residual", residual)
    T, H = residual.shape
    _check_tensor("y", y, residual.device)
    if y.shape != residual.shape:
        raise ValueError("y and residual must both be [T,H] (got %s, %s)" % (tuple(y.shape), tuple(residual.shape)))
    _check_weight("norm_weight", norm_weight, residual, H)
    if post_weight is not None:
        _check_weight("post_weight", post_weight, residual, H)
        if post_weight.dtype != norm_weight.dtype:
            raise TypeError("post_weight and norm_weight must have one type (got %s, %s)" % (post_weight.dtype, norm_weight.dtype))
    if gate is not None:
        _check_tensor("gate", gate, residual.device)
        _gate_kind(gate, T, H)
    return ResidualNormFunction.apply(y, residual, norm_weight, post_weight, gate,
                                      _check_scalar("residual_scale", residual_scale, False),
                                      _check_scalar("eps", eps, True))


def rms_norm(x, weight, *, eps=1e-6):
    """x / sqrt(mean(x^2) + eps) * weight, bf16: the norm before the first block.  x [T,H] and weight [H], each
    bf16 or float32; differentiable in both."""
    _check_stream("x", x)
    _check_weight("weight", weight, x, x.shape[1])
    return ResidualNormFunction.apply(None, x, weight, None, None, 1.0, _check_scalar("eps", eps, True))
