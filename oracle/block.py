"""Float64 references of the operators around the experts: the norms of a block.

Plain numpy, written from the formulas, sharing no code with the HIP path.  Each
gradient comes with the sum of the absolute terms it is made of, the scale that
float32 rounding errors are measured on.
"""

import numpy as np


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
