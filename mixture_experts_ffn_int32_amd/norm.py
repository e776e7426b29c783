"""Python binding of the norms around a block: ``residual_norm`` and ``rms_norm``.

Argument marshalling only; the kernels are those of csrc/norm.hip behind
hmm_residual_norm and hmm_residual_norm_backward.
"""

import ctypes
import functools
import math

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._bind import check_tensor, on_device, ptr, ready, stream_of

_MAX_H = 16384
_BF16 = (torch.bfloat16,)
_DTYPES = {torch.bfloat16: _lib.HMM_BF16, torch.float32: _lib.HMM_F32}
_EITHER = tuple(_DTYPES)


def _check_weight(name, w, H, device):
    check_tensor(name, w, _EITHER, (1,), device)
    if w.shape[0] != H:
        raise ValueError("%s must be [H] with H = %d (got %s)" % (name, H, tuple(w.shape)))


def _check_stream(name, r):
    check_tensor(name, r, _EITHER, (2,))
    H = r.shape[1]
    if H < 8 or H % 8 or H > _MAX_H:
        raise ValueError("%s must be [T,H] with H a multiple of 8 in [8, %d] (got %s)" % (name, _MAX_H, tuple(r.shape)))


def _check_scalar(name, v, positive):
    v = float(v)
    if not math.isfinite(v) or abs(v) > 3.4028234663852886e38 or (positive and v < 1.1754943508222875e-38):
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


@functools.lru_cache(maxsize=256)
def _problem(T, H, residual_dtype, weight_dtype, gate_kind, eps, scale):
    """(problem, backward workspace bytes)"""
    p = _lib.NormProblem(T, H, _DTYPES[residual_dtype], _DTYPES[weight_dtype], gate_kind, eps, scale)
    n = ctypes.c_size_t()
    _lib.check(_lib.load().hmm_residual_norm_backward_sizes(ctypes.byref(p), ctypes.byref(n)))
    return p, n.value


def _forward(y, residual, w, wp, g, prob, rstd_wanted):
    """(residual_out, normed, rstd) of arguments that are ready; residual_out None without y."""
    T, dev = residual.shape[0], residual.device
    out = None if y is None else torch.empty_like(residual)
    normed = torch.empty_like(residual, dtype=torch.bfloat16) if y is None else torch.empty_like(y)
    rstd = torch.empty((2, T), dtype=torch.float32, device=dev) if rstd_wanted else None
    if T > 0:
        with on_device(dev):
            _lib.check(_lib.load().hmm_residual_norm(prob, ptr(y), ptr(residual), ptr(w), ptr(wp), ptr(g), ptr(out),
                                                     ptr(normed), ptr(rstd), stream_of(dev)))
    return out, normed, rstd


class ResidualNormFunction(torch.autograd.Function):
    """Forward calls hmm_residual_norm; backward calls hmm_residual_norm_backward.  y None: the norm alone."""

    @staticmethod
    def forward(ctx, y, residual, norm_weight, post_weight, gate, prob, work_bytes):
        y, r, w, wp, g = (None if t is None else ready(t) for t in (y, residual, norm_weight, post_weight, gate))
        out, normed, rstd = _forward(y, r, w, wp, g, prob, True)
        ctx.set_materialize_grads(False)
        ctx.prob, ctx.work_bytes = prob, work_bytes
        ctx.save_for_backward(y, r if y is None else out, w, wp, g, rstd)
        return normed if y is None else (out, normed)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        d_out, d_normed = grads if len(grads) == 2 else (None, grads[0])
        if d_out is None and d_normed is None:
            return (None,) * 7
        y, r, w, wp, g, rstd = ctx.saved_tensors
        dev = r.device
        d_out = None if d_out is None else ready(d_out, r.dtype)
        d_normed = None if d_normed is None else ready(d_normed, torch.bfloat16)
        dy, dr, dw, dwp, dg = (None if t is None else torch.empty_like(t) for t in (y, r, w, wp, g))
        if r.shape[0] == 0:
            for t in (dw, dwp, dg):
                if t is not None:
                    t.zero_()
        else:
            work = torch.empty(ctx.work_bytes, dtype=torch.uint8, device=dev)
            with on_device(dev):
                _lib.check(_lib.load().hmm_residual_norm_backward(
                    ctx.prob, ptr(d_out), ptr(d_normed), ptr(y), ptr(r), ptr(w), ptr(wp), ptr(g), ptr(rstd), ptr(dy),
                    ptr(dr), ptr(dw), ptr(dwp), ptr(dg), ptr(work), ctx.work_bytes, stream_of(dev)))
        return dy, dr, dw, dwp, dg, None, None


def _call(y, residual, norm_weight, post_weight, gate, kind, scale, eps):
    T, H = residual.shape
    prob, work_bytes = _problem(T, H, residual.dtype, norm_weight.dtype, kind, eps, scale)
    tensors = (y, residual, norm_weight, post_weight, gate)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return ResidualNormFunction.apply(*tensors, prob, work_bytes)
    out, normed, _ = _forward(*(None if t is None else ready(t) for t in tensors), prob, False)
    return normed if y is None else (out, normed)


def residual_norm(y, residual, norm_weight, *, post_weight=None, gate=None, residual_scale=1.0, eps=1e-6):
    """(residual_out, normed): the norm after a block, its gate, the residual sum and the next block's norm, fused.

    With y bf16 [T,H] the block's output and residual [T,H] (bf16 or float32) the stream before it:
    u = y / sqrt(mean(y^2) + eps) (u = y without ``post_weight``);
    residual_out = residual + residual_scale * gate * post_weight * u, rounded to the residual's type;
    normed = residual_out / sqrt(mean(residual_out^2) + eps) * norm_weight, bf16, of the stored residual_out.
    norm_weight and post_weight are [H], both bf16 or both float32; gate is bf16 and multiplies per channel
    ([H]), per token ([T,1]) or per element ([T,H]).  Sums are float32: a row whose sum of squares is
    infinite has 1 / sqrt = 0.  Differentiable in all five tensors, in reverse mode.
    """
    _check_stream("residual", residual)
    T, H = residual.shape
    dev = residual.device
    check_tensor("y", y, _BF16, (2,), dev)
    if y.shape != residual.shape:
        raise ValueError("y and residual must both be [T,H] (got %s, %s)" % (tuple(y.shape), tuple(residual.shape)))
    _check_weight("norm_weight", norm_weight, H, dev)
    if post_weight is not None:
        _check_weight("post_weight", post_weight, H, dev)
        if post_weight.dtype != norm_weight.dtype:
            raise TypeError("post_weight and norm_weight must have one type (got %s, %s)" % (post_weight.dtype, norm_weight.dtype))
    if gate is not None:
        check_tensor("gate", gate, _BF16, (1, 2), dev)
    return _call(y, residual, norm_weight, post_weight, gate, _gate_kind(gate, T, H),
                 _check_scalar("residual_scale", residual_scale, False), _check_scalar("eps", eps, True))


def rms_norm(x, weight, *, eps=1e-6):
    """x / sqrt(mean(x^2) + eps) * weight, bf16: the norm before the first block.  x [T,H] and weight [H], each
    bf16 or float32; differentiable in both, in reverse mode."""
    _check_stream("x", x)
    _check_weight("weight", weight, x.shape[1], x.device)
    return _call(None, x, weight, None, None, _lib.HMM_GATE_NONE, 1.0, _check_scalar("eps", eps, True))
