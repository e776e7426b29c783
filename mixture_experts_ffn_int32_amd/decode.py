"""Python binding of the layer for a few tokens: ``moe_decode``.

Argument marshalling only; the kernels are those of csrc/decode.hip behind hmm_moe_decode.
"""

import ctypes
import functools

import torch

from . import _lib
from ._bind import check_tensor, on_device, ptr, ready, refuse_gradients, stream_of

_BF16 = (torch.bfloat16,)


@functools.lru_cache(maxsize=256)
def _problem(T, H, I, E, K, weight_dtype, router_dtype, flags):
    """(problem, workspace bytes)"""
    p = _lib.DecodeProblem(T, H, I, E, K, weight_dtype, router_dtype, flags)
    n = ctypes.c_size_t()
    _lib.check(_lib.load().hmm_moe_decode_sizes(ctypes.byref(p), ctypes.byref(n)))
    return p, n.value


def moe_decode(x, up_proj_weight, down_proj_weight, *, topk_ids=None, topk_weights=None, router_weight=None, top_k=None,
               renormalize=True, up_descale=None, down_descale=None):
    """A whole mixture-of-experts layer for at most 64 tokens, without gradients (serving).

    x is bf16 [T,H].  Either ``router_weight`` [E,H] (bf16 or float32) and ``top_k`` are given: the experts are
    the top_k largest logits x . router_weight^T (summed in 64 bits, ties to the lower expert), their weights the
    softmax over the chosen (``renormalize``) or over all experts, and the call returns (y, topk_ids, topk_weights).
    Or ``topk_ids`` [T,K] (int32 or int64; ids outside [0, E) are dropped) and ``topk_weights`` [T,K] are, and it
    returns y.  up_proj_weight [E,H,2I] and down_proj_weight [E,I,H] are bf16, as hyper_mega_moe takes them; or
    the uint8 E4M3 codes [E,2I,H] and [E,H,I] with ``up_descale`` [E,2I/128,H/128] and ``down_descale``
    [E,H/128,I/128] that quantize_block makes of them.  The weights must be contiguous: nothing of their size is
    copied.  For more tokens use hyper_mega_moe.
    """
    check_tensor("x", x, _BF16, (2,))
    T, H = x.shape
    dev = x.device
    fp8 = up_descale is not None or down_descale is not None
    if fp8 and (up_descale is None or down_descale is None):
        raise ValueError("up_descale and down_descale go together")
    wt = (torch.uint8,) if fp8 else _BF16
    check_tensor("up_proj_weight", up_proj_weight, wt, (3,), dev)
    check_tensor("down_proj_weight", down_proj_weight, wt, (3,), dev)
    E = up_proj_weight.shape[0]
    I = down_proj_weight.shape[2 if fp8 else 1]
    up, down = ((E, 2 * I, H), (E, H, I)) if fp8 else ((E, H, 2 * I), (E, I, H))
    if up_proj_weight.shape != up or down_proj_weight.shape != down:
        raise ValueError("up_proj_weight and down_proj_weight must be %s (got %s, %s, H=%d)"
                         % ("[E,2I,H] and [E,H,I]" if fp8 else "[E,H,2I] and [E,I,H]", tuple(up_proj_weight.shape),
                            tuple(down_proj_weight.shape), H))
    if not up_proj_weight.is_contiguous() or not down_proj_weight.is_contiguous():
        raise ValueError("up_proj_weight and down_proj_weight must be contiguous")
    if fp8:
        for name, t, shape in (("up_descale", up_descale, (E, 2 * I // 128, H // 128)),
                               ("down_descale", down_descale, (E, H // 128, I // 128))):
            check_tensor(name, t, (torch.float32,), (3,), dev)
            if t.shape != shape:
                raise ValueError("%s must be %s (got %s)" % (name, shape, tuple(t.shape)))
    routed = router_weight is not None
    rdt = _lib.HMM_BF16
    if routed:
        if topk_ids is not None or topk_weights is not None:
            raise ValueError("give router_weight and top_k, or topk_ids and topk_weights")
        if not isinstance(top_k, int) or isinstance(top_k, bool):
            raise TypeError("top_k must be an int (got %r)" % (top_k,))
        K = top_k
        check_tensor("router_weight", router_weight, (torch.bfloat16, torch.float32), (2,), dev)
        if router_weight.shape != (E, H):
            raise ValueError("router_weight must be [E,H] = %s (got %s)" % ((E, H), tuple(router_weight.shape)))
        if K > E:
            raise ValueError("top_k = %d experts a token of E = %d" % (K, E))
        if router_weight.dtype == torch.float32:
            rdt = _lib.HMM_F32
    else:
        if topk_ids is None or topk_weights is None or top_k is not None:
            raise ValueError("give router_weight and top_k, or topk_ids and topk_weights")
        check_tensor("topk_ids", topk_ids, (torch.int32, torch.int64), (2,), dev)
        check_tensor("topk_weights", topk_weights, (torch.float32, torch.bfloat16, torch.float16, torch.float64), (2,), dev)
        if topk_ids.shape[0] != T or topk_weights.shape != topk_ids.shape:
            raise ValueError("topk_ids and topk_weights must both be [T,K] with T = %d (got %s, %s)"
                             % (T, tuple(topk_ids.shape), tuple(topk_weights.shape)))
        K = topk_ids.shape[1]
    refuse_gradients("moe_decode has no gradient: use hyper_mega_moe, or call it under torch.no_grad()", x, up_proj_weight,
                     down_proj_weight, router_weight, topk_weights, up_descale, down_descale)
    prob, nbytes = _problem(T, H, I, E, K, _lib.HMM_FP8_E4M3_BLOCK if fp8 else _lib.HMM_BF16, rdt,
                            _lib.HMM_DECODE_RENORMALIZE if renormalize else 0)
    x = ready(x)
    if routed:
        wr = ready(router_weight)
        ids = torch.empty((T, K), dtype=torch.int32, device=dev)
        w = torch.empty((T, K), dtype=torch.float32, device=dev)
    else:
        wr = None
        if topk_ids.dtype == torch.int64:  # an id past 32 bits must not wrap into range
            topk_ids = topk_ids.clamp(-1, E)
        ids, w = ready(topk_ids, torch.int32), ready(topk_weights, torch.float32)
    ud, dd = (ready(up_descale), ready(down_descale)) if fp8 else (None, None)
    y = torch.empty_like(x)
    if T > 0:
        work = x.new_empty(nbytes // 2)  # nbytes is a multiple of 256
        with on_device(dev):
            _lib.check(_lib.load().hmm_moe_decode(prob, ptr(x), ptr(wr), ptr(ids), ptr(w), ptr(up_proj_weight), ptr(ud),
                                                  ptr(down_proj_weight), ptr(dd), ptr(y), ptr(work), nbytes, stream_of(dev)))
    return (y, ids, w) if routed else y
