"""Float64 references of the operators around the experts: the norms of a block, the E4M3
product with 128 x 128 block scales, and the layer for a few tokens.

Plain numpy, written from the formulas, sharing no code with the HIP path.  Each
gradient comes with the sum of the absolute terms it is made of, the scale that
float32 rounding errors are measured on.
"""

import numpy as np

from .quant import round_e4m3

GROUP = 128


def rms(v, eps):
    """1 / sqrt(mean(v^2) + eps) per row, [T, 1]."""
    return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def residual_sum(y, r, wp, gate, scale, eps):
    """The unrounded residual_out, and the sum of its absolute terms."""
    z = y * (rms(y, eps) * wp if wp is not None else 1.0) * (1.0 if gate is None else gate)
    return r + scale * z, np.abs(r) + np.abs(scale * z)


def residual_norm_grads(tr, dn, y, rs, w, wp, gate, scale, eps):
    """Gradients at the stored stream rs: {name: (value, absolute scale)}.

    y None: the norm alone.  tr or dn may be zero arrays."""
    rho = rms(rs, eps)
    a = dn * w
    m = np.mean(a * rs, axis=1, keepdims=True)
    ma = np.mean(np.abs(a * rs), axis=1, keepdims=True)
    t = tr + rho * a - rs * rho ** 3 * m
    ta = np.abs(tr) + np.abs(rho * a) + np.abs(rs) * rho ** 3 * ma
    out = {"d_residual": (t, ta), "d_norm_weight": (np.sum(dn * rs * rho, axis=0), np.sum(np.abs(dn * rs * rho), axis=0))}
    if y is None:
        return out
    rho_y = rms(y, eps) if wp is not None else np.ones((y.shape[0], 1))
    wpv = 1.0 if wp is None else wp
    g = 1.0 if gate is None else gate
    u = y * rho_y
    b, ba = scale * t * g * wpv, np.abs(scale * g * wpv) * ta
    if wp is None:
        out["d_y"] = (b, ba)
    else:
        out["d_y"] = (rho_y * b - y * rho_y ** 3 * np.mean(b * y, axis=1, keepdims=True),
                      rho_y * ba + np.abs(y) * rho_y ** 3 * np.mean(ba * np.abs(y), axis=1, keepdims=True))
        out["d_post_weight"] = (np.sum(scale * t * g * u, axis=0), np.sum(np.abs(scale * g * u) * ta, axis=0))
    if gate is not None:
        dg, dga = scale * t * wpv * u, np.abs(scale * wpv * u) * ta
        if gate.shape == y.shape:
            out["d_gate"] = (dg, dga)
        elif gate.ndim == 1:
            out["d_gate"] = (dg.sum(axis=0), dga.sum(axis=0))
        else:
            out["d_gate"] = (dg.sum(axis=1, keepdims=True), dga.sum(axis=1, keepdims=True))
    return out


def e4m3_values(codes):
    """E4M3 bytes as the values they stand for (OCP e4m3fn: bias 7, no infinity, 0x7f is NaN)."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7, -v, v)


def _quantize(v):
    """E4M3 values and float32 descales of rows v [n, L] (float32), one scale per row: 448 times the rounded reciprocal
    of the largest, at most the largest float32; 1 for a row of zeros."""
    v = np.asarray(v, np.float32)
    m = np.max(np.abs(v), axis=-1)
    with np.errstate(divide="ignore", over="ignore"):
        s = np.minimum((np.float32(1.0) / m).astype(np.float32) * np.float32(448.0), np.finfo(np.float32).max)
    s = np.where(m > 0, s, np.float32(1.0)).astype(np.float32)
    q = round_e4m3((v * s[..., None]).astype(np.float32).astype(np.float64))
    return q, (np.float32(1.0) / s).astype(np.float32)


def quantize_rows_block(x):
    """(E4M3 values [T,H], float32 descales [T,H/128]) of x [T,H]: one scale per token and group of 128."""
    T, H = x.shape
    q, d = _quantize(np.asarray(x, np.float32).reshape(T * (H // GROUP), GROUP))
    return q.reshape(T, H), d.reshape(T, H // GROUP)


def quantize_block(w):
    """(E4M3 values [N,H], float32 descales [ceil(N/128), H/128]) of w [H,N], one scale per block."""
    H, N = w.shape
    nb, hb = (N + GROUP - 1) // GROUP, H // GROUP
    t = np.zeros((nb * GROUP, H), np.float32)
    t[:N] = np.asarray(w, np.float32).T
    q, d = _quantize(t.reshape(nb, GROUP, hb, GROUP).transpose(0, 2, 1, 3).reshape(nb * hb, GROUP * GROUP))
    q = q.reshape(nb, hb, GROUP, GROUP).transpose(0, 2, 1, 3).reshape(nb * GROUP, H)[:N]
    return q, d.reshape(nb, hb)


def block_product(xv, xs, wv, ws):
    """y of token values xv [T,H] and descales xs [T,H/128], weight values wv [N,H] and block descales ws.

    Returns (y, largest |x| times largest |w| of each group with its scales, summed; sum of absolute scaled groups)."""
    T, H = xv.shape
    N = wv.shape[0]
    y, big, sabs = (np.zeros((T, N)) for _ in range(3))
    rep = np.arange(N) // GROUP
    for g in range(H // GROUP):
        k = slice(g * GROUP, (g + 1) * GROUP)
        s = xs[:, g].astype(np.float64)[:, None] * ws[rep, g].astype(np.float64)[None]
        p = xv[:, k] @ wv[:, k].T
        y += s * p
        sabs += np.abs(s * p)
        big += s * np.abs(xv[:, k]).max(axis=1)[:, None] * np.abs(wv[:, k]).max(axis=1)[None]
    return y, big, sabs


def route(x, wr, K, renormalize):
    """The K largest logits of each token (ties to the lower expert) and their softmax weights."""
    logits = x @ wr.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :K]
    e = np.exp(logits - logits.max(axis=1, keepdims=True))
    p = np.take_along_axis(e, ids, axis=1)
    return ids.astype(np.int32), p / (p if renormalize else e).sum(axis=1, keepdims=True)


def moe(x, ids, weights, up, down, eh, ea, eo):
    """y of the layer for a few tokens and the bound of its float32 error before y's rounding.

    up(e) [H,2I] and down(e) [I,H] give an expert's matrices.  eh: relative error of the up-projection's sums
    (of the sum of absolute products), ea: of a, eo: of the down-projection's and the weighted sums."""
    T, K = ids.shape
    y = np.zeros_like(x)
    dev = np.zeros_like(x)
    for t in range(T):
        for k in range(K):
            e = ids[t, k]
            try:
                W1, W2 = up(e), down(e)
            except IndexError:
                continue
            I = W2.shape[0]
            h, ha = x[t] @ W1, eh * (np.abs(x[t]) @ np.abs(W1))
            g, u, dg, du = h[:I], h[I:], ha[:I], ha[I:]
            s = 1.0 / (1.0 + np.exp(-g))
            a = g * s * u
            # |d silu| <= 1.1; second order terms are far below the bound's slack
            da = 1.1 * dg * np.abs(u) + np.abs(g * s) * du + ea * np.abs(a)
            y[t] += weights[t, k] * (a @ W2)
            dev[t] += np.abs(weights[t, k]) * (da @ np.abs(W2) + eo * (np.abs(a) @ np.abs(W2)))
    return y, dev
