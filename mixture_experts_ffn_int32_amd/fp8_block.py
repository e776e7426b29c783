"""Python binding of the E4M3 product with 128 x 128 block scales: ``quantize_block``,
``quantize_rows_block``, ``matmul_fp8_block`` and the differentiable ``linear_fp8_block``.

Argument marshalling only; the kernels are those of csrc/fp8_block.hip behind
hmm_quant_block, hmm_matmul_fp8_block, hmm_linear_fp8_block and hmm_linear_fp8_block_grad.
"""

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._bind import check_tensor, on_device, ptr, ready, refuse_gradients, stream_of

GROUP = 128
_BF16, _U8, _F32 = (torch.bfloat16,), (torch.uint8,), (torch.float32,)


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
    _lib.check(_lib.load().hmm_quant_block(ptr(w), E, H, N, ptr(qt), ptr(q), ptr(ds), stream_of(dev)))
    return qt, q, ds


def quantize_block(w):
    """E4M3 codes of a weight, one scale per block of 128 x 128, for linear_fp8_block and moe_decode.

    w bf16 [H,N] or [E,H,N], H a multiple of 128 and N of 16 (a last block of columns may be narrower).
    Returns (codes uint8 [(E,) N, H], descale float32 [(E,) ceil(N/128), H/128]): the codes are transposed, so
    that the contraction is contiguous.  Per block, in float32: scale = 448 * (1 / max|block|) (1 for
    zeros), code = E4M3 of w * scale, descale = 1 / scale.  Both are detached from w."""
    check_tensor("w", w, _BF16, (2, 3))
    _widths(w.shape[-2], w.shape[-1], 16)
    if w.dim() == 3 and w.shape[0] < 1:
        raise ValueError("w must hold at least one matrix (got %s)" % (tuple(w.shape),))
    with on_device(w.device):
        qt, _, ds = _quant(ready(w.detach() if w.dim() == 3 else w.detach()[None]), False)
    return (qt, ds) if w.dim() == 3 else (qt[0], ds[0])


def quantize_rows_block(x):
    """The tokens' side: (codes uint8 [T,H], descale float32 [T,H/128]) of x bf16 [T,H], quantize_block's rule per token
    and group of 128, as linear_fp8_block applies it; detached from x."""
    check_tensor("x", x, _BF16, (2,))
    T, H = x.shape
    _widths(GROUP, H, GROUP)
    x = ready(x.detach())
    q = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    d = torch.empty((T, H // GROUP), dtype=torch.float32, device=x.device)
    with on_device(x.device):
        _lib.check(_lib.load().hmm_quant_rows_block(ptr(x), T, H, ptr(q), ptr(d), stream_of(x.device)))
    return q, d


def _check_codes(codes, descale, H, device):
    check_tensor("codes", codes, _U8, (2,), device)
    check_tensor("descale", descale, _F32, (2,), device)
    N = codes.shape[0]
    _widths(H, N, 16)
    if codes.shape[1] != H or descale.shape != ((N + GROUP - 1) // GROUP, H // GROUP):
        raise ValueError("codes must be [N,H] and descale [ceil(N/128),H/128] (got %s, %s, H=%d)"
                         % (tuple(codes.shape), tuple(descale.shape), H))
    return N


def matmul_fp8_block(xq, xs, codes, descale):
    """y bf16 [T,N] of tokens (xq uint8 [T,H], xs float32 [T,H/128], as quantize_rows_block gives them) and a weight
    (codes uint8 [N,H], descale float32 [ceil(N/128),H/128], as quantize_block does).  It has no gradient."""
    check_tensor("xq", xq, _U8, (2,))
    T, H = xq.shape
    check_tensor("xs", xs, _F32, (2,), xq.device)
    N = _check_codes(codes, descale, H, xq.device)
    if xs.shape != (T, H // GROUP):
        raise ValueError("xs must be [T,H/128] (got %s, T=%d, H=%d)" % (tuple(xs.shape), T, H))
    refuse_gradients("matmul_fp8_block has no gradient: use linear_fp8_block, or call it under torch.no_grad()", xs, descale)
    dev = xq.device
    with on_device(dev):
        xq, xs, codes, descale = (ready(t) for t in (xq, xs, codes, descale))
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        _lib.check(_lib.load().hmm_matmul_fp8_block(ptr(xq), ptr(xs), ptr(codes), ptr(descale), T, H, N, ptr(y),
                                                    stream_of(dev)))
    return y


@functools.lru_cache(maxsize=256)
def _sizes(T, H, N):
    """Workspace bytes of the forward and of the gradient."""
    fwd, grad = ctypes.c_size_t(), ctypes.c_size_t()
    _lib.check(_lib.load().hmm_linear_fp8_block_sizes(T, H, N, ctypes.byref(fwd), ctypes.byref(grad)))
    return fwd.value, grad.value


def _linear(x, codes, descale, N):
    T, H = x.shape
    dev = x.device
    lib = _lib.load()
    nbytes = _sizes(T, H, N)[0]
    y = x.new_empty((T, N))
    work = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _lib.check(lib.hmm_linear_fp8_block(ptr(x), ptr(codes), ptr(descale), T, H, N, ptr(y), ptr(work), nbytes, stream_of(dev)))
    return y


class LinearFp8BlockFunction(torch.autograd.Function):
    """Forward quantises the weight and calls hmm_linear_fp8_block; backward calls hmm_linear_fp8_block_grad."""

    @staticmethod
    def forward(ctx, x, weight):
        x_, w = ready(x), ready(weight)
        with on_device(x.device):
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
        with on_device(dev):
            dy = ready(dy, torch.bfloat16)
            dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if q is not None else None
            dw = torch.empty((H, N), dtype=torch.bfloat16, device=dev) if x is not None else None
            nbytes = _sizes(T, H, N)[1]
            work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            _lib.check(lib.hmm_linear_fp8_block_grad(ptr(dy), ptr(x), ptr(q), ptr(ds), T, H, N, ptr(dx), ptr(dw),
                                                     ptr(work), nbytes, stream_of(dev)))
        return dx, dw


def linear_fp8_block(x, weight):
    """y bf16 [T,N] = x . weight on E4M3: a dense projection with 128-deep scales.

    x bf16 [T,H] is quantised per token and group of 128 (quantize_rows_block's rule).  ``weight`` is either bf16
    [H,N], quantised per block of 128 x 128 in the call (H and N multiples of 128): then the call is differentiable in
    both, dx from the E4M3 codes of dy (per token and 128 of N) and of the weight, dw = x^T dy as a bf16 product, the
    quantisation's own derivative taken as 1.  Or a pair (codes, descale) from quantize_block (serving; N a multiple
    of 16): no gradient.  At most 16 tokens of a quantised weight take one launch."""
    check_tensor("x", x, _BF16, (2,))
    H = x.shape[1]
    if isinstance(weight, torch.Tensor):
        check_tensor("weight", weight, _BF16, (2,), x.device)
        if weight.shape[0] != H:
            raise ValueError("weight must be [H,N] with H = %d (got %s)" % (H, tuple(weight.shape)))
        _widths(H, weight.shape[1], GROUP)
        return LinearFp8BlockFunction.apply(x, weight)
    if not isinstance(weight, (tuple, list)) or len(weight) != 2:
        raise TypeError("weight must be a bf16 tensor [H,N] or a pair (codes, descale)")
    codes, descale = weight
    N = _check_codes(codes, descale, H, x.device)
    refuse_gradients("a quantised weight has no gradient: give the bf16 weight, or call under torch.no_grad()", x, descale)
    with on_device(x.device):
        return _linear(ready(x), ready(codes), ready(descale), N)
