"""moe_decode within bounds that follow from how its kernels split a contraction of length L.

A chain of n additions in float32 is off by at most n 2^-23 of its absolute sum (an addition of the matrix
instruction may cut instead of round).  bf16 weights: four waves take steps of 32 in turn, in the wide tiles two, so
a wave chains L / 2 products at most, and 4 sums meet at the end; in the down-projection every step is taken twice
(the activation's two halves): L.  E4M3 weights: a step's own products, 128 or twice that, then one scaling and one
addition a step, L / 64 / 4 of them at most, and 4 sums.  The activation: silu's exponential, reciprocal and products
16 2^-24, kept as two bf16, 2^-17; the weighted sum of K rows K + 1.  y is rounded once, 2^-8 of it.
That is a worst case, so the whole error's 2-norm is held to y's rounding as well.
"""

import numpy as np
import pytest
import torch

from _util import announce, to_f64
from test_gpu_decode import _layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


def _bounds(H, I, K, fp8):
    a = 16 * 2.0 ** -24 + 2.0 ** -17
    if fp8:
        return (128 + H / 128 + 6) * U, a, (256 + I / 128 + 6 + K + 1) * U
    return (H / 2 + 4) * U, a, (I + 4 + K + 1) * U


def _moe(x, ids, w, ref, E, eh, ea, eo):
    """y in float64 and the bound of its error before its rounding, expert by expert (no id occurs twice in a row)."""
    y, dev = np.zeros_like(x), np.zeros_like(x)
    for e in range(E):
        t, k = np.nonzero(ids == e)
        if t.size == 0:
            continue
        W1, W2 = ref[0](e), ref[1](e)
        I = W2.shape[0]
        h, ha = x[t] @ W1, eh * (np.abs(x[t]) @ np.abs(W1))
        g, u = h[:, :I], h[:, I:]
        s = g / (1.0 + np.exp(-g))
        # silu's derivative is at most 1.1; the errors' products are far below the bounds' slack
        da = 1.1 * ha[:, :I] * np.abs(u) + np.abs(s) * ha[:, I:] + ea * np.abs(s * u)
        y[t] += w[t, k, None] * (s * u @ W2)
        dev[t] += w[t, k, None] * ((da + eo * np.abs(s * u)) @ np.abs(W2))
    return y, dev


@pytest.mark.parametrize("T,H,I,E,K,fp8", [
    (1, 1024, 512, 16, 4, False), (4, 2048, 64, 4, 2, False), (64, 512, 1088, 8, 4, False),     # narrow tiles
    (16, 2112, 512, 130, 8, False), (64, 1088, 640, 108, 16, False),                            # wide, one and two row tiles
    (3, 1024, 256, 8, 3, True), (64, 1152, 384, 8, 4, True), (20, 640, 1280, 40, 2, True)])
def test_bounds(T, H, I, E, K, fp8):
    import mixture_experts_ffn_int32_amd as hmm
    announce("moe_decode bounds %s" % ((T, H, I, E, K, fp8),))
    x, weights, scales, ref = _layer(T, H, I, E, 13, fp8)
    g = torch.Generator().manual_seed(14)
    ids = torch.rand((T, E), generator=g).argsort(dim=1)[:, :K].int()
    w = torch.softmax(torch.randn((T, K), generator=g), dim=1)
    y = hmm.moe_decode(x.cuda(), *weights, topk_ids=ids.cuda(), topk_weights=w.cuda(), **scales)
    want, dev = _moe(x.float().numpy().astype(np.float64), ids.numpy(), w.numpy().astype(np.float64), ref, E,
                     *_bounds(H, I, K, fp8))
    err = np.abs(to_f64(y) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + dev), float(np.max(err - 2.0 ** -8 * np.abs(want) - dev))
    assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(want)
