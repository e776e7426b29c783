"""Python binding of the E4M3 product with 128 x 128 block scales: ``quantize_block``,
``quantize_rows_block``, ``matmul_fp8_block`` and the differentiable ``linear_fp8_block``.

Argument marshalling only; the kernels are those of csrc/fp8_block.hip behind
hmm_quant_block, hmm_matmul_fp8_block, hmm_linear_fp8_block and hmm_linear_fp8_block_grad.
"""

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .moe import _aligned, _ptr, _stream

GROUP = 128


def _tensor(name, t, dtype, dims, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be on a HIP device (got %s)" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.dim() not in dims:
        raise ValueError("%s must have %s dimensions (got %s)" % (name, " or ".join(map(str, dims)), tuple(t.shape)))


def _widths(H, N, step):
    if H < GROUP or H % GROUP or N < step or N % step:
        raise ValueError("H must be a positive multiple of %d and N of %d (got %d, %d)" % (GROUP, step, H, N))


def _quant(w, both):
    """codes_t, codes (None unless ``both``), descale of a contiguous w [E,H,N]."""
    E, H, N = w.shape
    dev = w.device
    qt = torch.empty((E, N, H), dtype=torch.uint8, device=dev)
    q = torch.empty((E, H, N), dtype=torch.uint8, device=dev) if both else None
    ds = torch.empty((E, (N + GROUP - 1) // GROUP, H // GROUP), dtype=torch.float32, device=dev)
    _lib.check(_lib.load().hmm_quant_block(_ptr(w), E, H, N, _ptr(qt), _ptr(q), _ptr(ds), _stream(dev)))
    return qt, q, ds


def quantize_block(w):
    """E4M3 codes of a weight, one scale per block of 128 x 128, for linear_fp8_block and moe_decode.

    w bf16 [H,N] or [E,H,N], H a multiple of 128 and N of 16 (a last block of columns may be narrower).
    Returns (codes uint8 [(E,) N, H], descale float32 [(E,) ceil(N/128), H/128]): the codes are transposed, so
    that the contraction is contiguous.  Per block, in float32: scale = 448 * (1 / max|block|) (1 for
    zeros), code = E4M3 of w * scale, descale = 1 / scale."""
    _tensor("w", w, torch.bfloat16, (2, 3))
    _widths(w.shape[-2], w.shape[-1], 16)
    if w.dim() == 3 and w.shape[0] < 1:
        raise ValueError("w must hold at least one matrix (got %s)" % (tuple(w.shape),))
    with torch.cuda.device(w.device):
        qt, _, ds = _quant(_aligned(w.detach() if w.dim() == 3 else w.detach()[None]), False)
    return (qt, ds) if w.dim() == 3 else (qt[0], ds[0])


def quantize_rows_block(x):
    """The tokens' side: (codes uint8 [T,H], descale float32 [T,H/128]) of x bf16 [T,H], quantize_block's rule per token
    and group of 128, as linear_fp8_block applies it."""
    _tensor("x", x, torch.bfloat16, (2,))
    T, H = x.shape
    _widths(GROUP, H, GROUP)
    x = _aligned(x.detach())
    q = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    d = torch.empty((T, H // GROUP), dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):
        _lib.check(_lib.load().hmm_quant_rows_block(_ptr(x), T, H, _ptr(q), _ptr(d), _stream(x.device)))
    return q, d


def _check_codes(codes, descale, H, device):
    _tensor("codes", codes, torch.uint8, (2,), device)
    _tensor("descale", descale, torch.float32, (2,), device)
    N = codes.shape[0]
    _widths(H, N, 16)
    if codes.shape[1] != H or tuple(descale.shape) != ((N + GROUP - 1) // GROUP, H // GROUP):
        raise ValueError("codes must be [N,H] and descale [ceil(N/128),H/128] (got %s, %s, H=%d)"
                         % (tuple(codes.shape), tuple(descale.shape), H))
    return N


def matmul_fp8_block(xq, xs, codes, descale):
    """y bf16 [T,N] of tokens (xq uint8 [T,H], xs float32 [T,H/128], as quantize_rows_block gives them) and a weight
    (codes uint8 [N,H], descale float32 [ceil(N/128),H/128], as quantize_block does)."""
    _tensor("xq", xq, torch.uint8, (2,))
    T, H = xq.shape
    _tensor("xs", xs, torch.float32, (2,), xq.device)
    N = _check_codes(codes, descale, H, xq.device)
    if tuple(xs.shape) != (T, H // GROUP):
        raise ValueError("xs must be [T,H/128] (got %s, T=%d, H=%d)" % (tuple(xs.shape), T, H))
    dev = xq.device
    with torch.cuda.device(dev):
        xq, xs, codes, descale = (_aligned(t) for t in (xq, xs, codes, descale))
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        _lib.check(_lib.load().hmm_matmul_fp8_block(_ptr(xq), _ptr(xs), _ptr(codes), _ptr(descale), T, H, N, _ptr(y),
                                                    _stream(dev)))
    return y


def _linear(x, codes, descale, N):
    T, H = x.shape
    dev = x.device
    lib = _lib.load()
    fwd, grad = ctypes.c_size_t(), ctypes.c_size_t()
    _lib.check(lib.hmm_linear_fp8_block_sizes(T, H, N, ctypes.byref(fwd), ctypes.byref(grad)))
    y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    work = torch.empty(fwd.value, dtype=torch.uint8, device=dev) if fwd.value else None
    _lib.check(lib.hmm_linear_fp8_block(_ptr(x), _ptr(codes), _ptr(descale), T, H, N, _ptr(y), _ptr(work), fwd.value,
                                        _stream(dev)))
    return y


class LinearFp8BlockFunction(torch.autograd.Function):
    """Forward quantises the weight and calls hmm_linear_fp8_block; backward calls hmm_linear_fp8_block_grad."""

    @staticmethod
    def forward(ctx, x, weight):
        x_, w = _aligned(x), _aligned(weight)
        with torch.cuda.device(x.device):
            qt, q, ds = _quant(w[None], ctx.needs_input_grad[0])
            y = _linear(x_, qt, ds, w.shape[1])
        ctx.save_for_backward(x_ if ctx.needs_input_grad[1] else None, q, ds)
        ctx.dims = (x.shape[0],) + tuple(w.shape)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, q, ds = ctx.saved_tensors
        T, H, N = ctx.dims
        dev = dy.device
        lib = _lib.load()
        with torch.cuda.device(dev):
            dy = _aligned(dy, torch.bfloat16)
            dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if q is not None else None
            dw = torch.empty((H, N), dtype=torch.bfloat16, device=dev) if x is not None else None
            fwd, grad = ctypes.c_size_t(), ctypes.c_size_t()
            _lib.check(lib.hmm_linear_fp8_block_sizes(T, H, N, ctypes.byref(fwd), ctypes.byref(grad)))
            work = torch.empty(grad.value, dtype=torch.uint8, device=dev)
            _lib.check(lib.hmm_linear_fp8_block_grad(_ptr(dy), _ptr(x), _ptr(q), _ptr(ds), T, H, N, _ptr(dx), _ptr(dw),
                                                     _ptr(work), grad.value, _stream(dev)))
        return dx, dw


def linear_fp8_block(x, weight):
    """y bf16 [T,N] = x . weight on E4M3: a dense projection with 128-deep scales.

    x bf16 [T,H] is quantised per token and group of 128 (quantize_rows_block's rule).  ``weight`` is either bf16
    [H,N], quantised per block of 128 x 128 in the call (H and N multiples of 128): then the call is differentiable in
    both, dx from the E4M3 codes of dy (per token and 128 of N) and of the weight, dw = x^T dy as a bf16 product, the
    quantisation's own derivative taken as 1.  Or a pair (codes, descale) from quantize_block (serving; N a multiple
    of 16): no gradient.  At most 64 tokens of a quantised weight take one launch."""
    _tensor("x", x, torch.bfloat16, (2,))
    H = x.shape[1]
    if isinstance(weight, torch.Tensor):
        _tensor("weight", weight, torch.bfloat16, (2,), x.device)
        if weight.shape[0] != H:
            raise ValueError("weight must be [H,N] with H = %d (got %s)" % (H, tuple(weight.shape)))
        _widths(H, weight.shape[1], GROUP)
        return LinearFp8BlockFunction.apply(x, weight)
    if not isinstance(weight, (tuple, list)) or len(weight) != 2:
        raise TypeError("weight must be a bf16 tensor [H,N] or a pair (codes, descale)")
    codes, descale = weight
    N = _check_codes(codes, descale, H, x.device)
    if torch.is_grad_enabled() and x.requires_grad:
        raise ValueError("a quantised weight has no gradient: give the bf16 weight, or call under torch.no_grad()")
    with torch.cuda.device(x.device):
        return _linear(_aligned(x), _aligned(codes), _aligned(descale), N)
