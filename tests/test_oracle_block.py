"""The float64 references of oracle/block.py against differences of their own forward."""

import numpy as np
import pytest

from oracle import block


def _loss(y, r, w, wp, g, scale, eps, tr, dn):
    rs, _ = block.residual_sum(y, r, wp, g, scale, eps)
    return np.sum(tr * rs) + np.sum(dn * rs * block.rms(rs, eps) * w)


@pytest.mark.parametrize("gate,post", [("none", True), ("token", True), ("channel", True), ("full", True), ("full", False)])
def test_norm_gradients_against_differences(gate, post):
    rng = np.random.default_rng(3)
    T, H, scale, eps = 3, 8, 0.7, 1e-3
    v = {"y": rng.standard_normal((T, H)), "r": rng.standard_normal((T, H)), "w": rng.standard_normal(H),
         "wp": rng.standard_normal(H) if post else None,
         "g": {"none": None, "token": rng.standard_normal((T, 1)), "channel": rng.standard_normal(H),
               "full": rng.standard_normal((T, H))}[gate]}
    tr, dn = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    rs, _ = block.residual_sum(v["y"], v["r"], v["wp"], v["g"], scale, eps)
    grads = block.residual_norm_grads(tr, dn, v["y"], rs, v["w"], v["wp"], v["g"], scale, eps)
    names = {"y": "d_y", "r": "d_residual", "w": "d_norm_weight", "wp": "d_post_weight", "g": "d_gate"}
    h = 1e-5
    for k, name in names.items():
        if v[k] is None:
            assert name not in grads
            continue
        got, scale_of = grads[name]
        assert got.shape == v[k].shape
        assert np.all(np.abs(got) <= scale_of * (1 + 1e-12))
        num = np.empty_like(v[k])
        for i in np.ndindex(*v[k].shape):
            lo, hi = (dict(v, **{k: v[k].copy()}) for _ in range(2))
            lo[k][i] -= h
            hi[k][i] += h
            num[i] = (_loss(**hi, scale=scale, eps=eps, tr=tr, dn=dn) - _loss(**lo, scale=scale, eps=eps, tr=tr, dn=dn)) / (2 * h)
        # central differences: h^2 f'''/6 (f''' of order 1e2 here) plus 1e-16 / h of rounding
        np.testing.assert_allclose(got, num, rtol=1e-6, atol=1e-6)
