"""The norms' gradients at the ends of what the entry points accept: eps down to the smallest normal
float32, rows of zeros, rows of 1e-18 and rows whose squares come close to float32's largest value.

Tolerance: as for ordinary rows, an output is off by its rounding and by at most C roundings of 2^-24 of
the sum of its absolute terms (float64 reference, oracle/block.py).  That holds here as there as long as
no intermediate value leaves float32's normal range: the normalised rows r' rho and y rho_y are at most
sqrt(H), whatever rho is.  A row sum chains at most 32 elements a thread (four chunks of 8), 6 steps
across a wave and 8 waves, a gradient two of them and a few products: about 100 roundings; a column
sum adds its T rows and at most 64 partial sums in turn besides: C = 256 and 256 + T are more than both.
"""

import numpy as np
import pytest
import torch

from _util import announce, to_f64
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _f(t):
    return None if t is None else to_f64(t.detach())


def _close(got, ref, scale, c, what):
    r = to_f64(got.detach())
    assert r.shape == ref.shape, what
    tol = torch.finfo(got.dtype).eps / 2 * np.abs(ref) + c * U * scale
    err = np.abs(r - ref)
    assert np.all(err <= tol), (what, float(np.nanmax(err - tol)), float(np.nanmax(err)), bool(np.isnan(r).any()))


def _rows(g, T, H, rms):
    """Row t has rms[t % len(rms)]; a part of it is the same in every row, so that gradients project on it."""
    return torch.randn((T, H), generator=g) * torch.tensor([rms[t % len(rms)] for t in range(T)])[:, None]


# rms of the rows, eps: zeros and ordinary rows with an eps whose power -3/2 passes float32; tiny rows with the
# smallest eps; rows whose rho^3 is subnormal or zero in float32
RANGES = [((0.0, 1.0), 1e-27), ((0.0, 1.0), 1e-30), ((1e-18, 0.0, 3e-19), 1.2e-38), ((1e14, 1.0, 1e15), 1e-6),
          ((1e16, 0.0, 1e17), 1e-5)]


@pytest.mark.parametrize("T,H,dt", [(5, 264, "f32"), (6, 1024, "bf16"), (4, 1536, "f32"), (3, 2048, "bf16"), (5, 4096, "f32"),
                                    (4, 7168, "bf16"), (3, 8200, "f32")])
@pytest.mark.parametrize("rms,eps", RANGES)
def test_rms_norm(T, H, dt, rms, eps):
    import mixture_experts_ffn_int32_amd as hmm
    announce("rms_norm range T=%d H=%d %s rms=%s eps=%g" % (T, H, dt, rms, eps))
    g = torch.Generator().manual_seed(3)
    dn = torch.randn((T, H), generator=g)
    x = _rows(g, T, H, rms)
    x += 0.5 * dn * torch.tensor([rms[t % len(rms)] for t in range(T)])[:, None]  # a projection that counts
    x, dn = x.to(TYPES[dt]).cuda().requires_grad_(True), dn.bfloat16().cuda()
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(TYPES[dt]).cuda().requires_grad_(True)
    n = hmm.rms_norm(x, w, eps=eps)
    dx, dw = torch.autograd.grad(n, (x, w), dn)
    xf, wf, e = _f(x), _f(w), float(np.float32(eps))
    ref = xf * block.rms(xf, e) * wf
    _close(n, ref, np.abs(ref), 256, "normed")
    want = block.residual_norm_grads(np.zeros_like(xf), _f(dn), None, xf, wf, None, None, 1.0, e)
    _close(dx, *want["d_residual"], 256, "dx")
    _close(dw, *want["d_norm_weight"], 256 + T, "dw")


@pytest.mark.parametrize("T,H,res,wt,gate", [(5, 264, "f32", "f32", "channel"), (6, 1024, "bf16", "f32", "token"),
                                             (4, 2048, "bf16", "bf16", "full"), (7, 7168, "f32", "bf16", "none")])
@pytest.mark.parametrize("rms_y,rms_r,eps", [
    ((0.0, 1.0), (1.0, 0.0), 1e-30),       # a block that gave nothing, and a row of the stream that is zero
    ((0.0,), (0.0, 1.0), 1e-30),           # both zero in one row
    ((1e15, 1.0), (1.0,), 1e-6),           # a block's large rows, normalised by the post-norm
    ((1.0,), (1e15, 1.0, 1e16), 1e-6)])    # a stream's large rows
def test_residual_norm(T, H, res, wt, gate, rms_y, rms_r, eps):
    import mixture_experts_ffn_int32_amd as hmm
    announce("residual_norm range T=%d H=%d %s %s %s y=%s r=%s eps=%g" % (T, H, res, wt, gate, rms_y, rms_r, eps))
    g = torch.Generator().manual_seed(4)

    def rnd(*shape):
        return torch.randn(shape, generator=g)
    tr, dn = rnd(T, H), rnd(T, H)
    y, r = _rows(g, T, H, rms_y), _rows(g, T, H, rms_r)
    y += 0.5 * tr * torch.tensor([rms_y[t % len(rms_y)] for t in range(T)])[:, None]
    r += 0.5 * dn * torch.tensor([rms_r[t % len(rms_r)] for t in range(T)])[:, None]
    gv = {"none": None, "token": rnd(T, 1), "channel": rnd(H), "full": rnd(T, H)}[gate]
    v = {"y": y.bfloat16(), "residual": r.to(TYPES[res]), "norm_weight": (1 + 0.3 * rnd(H)).to(TYPES[wt]),
         "post_weight": (1 + 0.3 * rnd(H)).to(TYPES[wt]), "gate": None if gv is None else gv.bfloat16()}
    v = {k: None if t is None else t.cuda().requires_grad_(True) for k, t in v.items()}
    tr, dn = tr.to(TYPES[res]).cuda(), dn.bfloat16().cuda()
    out, n = hmm.residual_norm(v["y"], v["residual"], v["norm_weight"], post_weight=v["post_weight"], gate=v["gate"], eps=eps)
    names = [k for k in v if v[k] is not None]
    e = float(np.float32(eps))
    for d_out in (tr, None):  # without a gradient of the stream, what the norm gives stands alone
        use = ((out, n), (tr, dn)) if d_out is not None else (n, dn)
        grads = torch.autograd.grad(use[0], [v[k] for k in names], use[1], retain_graph=True)
        f = {k: _f(t) for k, t in v.items()}
        want = block.residual_norm_grads(_f(tr) if d_out is not None else np.zeros((T, H)), _f(dn), f["y"], _f(out),
                                         f["norm_weight"], f["post_weight"], f["gate"], 1.0, e)
        for k, t in zip(names, grads):
            _close(t, *want["d_" + k], 256 + T, ("d_" + k, d_out is not None))
