"""The norms with more rows than their launches take at once: a wave or a workgroup walks several rows, the next
one loaded ahead, so a row must not reach into another.  One case for each number of threads a row.

At once: the forward takes 2^19 threads' rows (8192 of up to 1024 elements, 2730 of 1536, 2048 of up to 4096, 1024 of
8192, 512 above), the backward 2048 rows of up to 1024 elements, 768 of up to 2048, 512 of up to 4096, 256 above.
Tolerances: an output's own rounding and C roundings of 2^-24 of the sum of its absolute terms.  A row sum chains at
most 32 elements a thread, 6 steps across a wave and 16 waves, a gradient two of them and a few products: about 120,
C = 256.  A column sum adds a walker's rows, four walkers, and 768 / 16 + 16 partial rows besides: C = 256 + T.
"""

import ctypes

import numpy as np
import pytest
import torch

from _util import announce, to_f64
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _close(got, ref, scale, c, what):
    r = to_f64(got.detach())
    assert r.shape == ref.shape, what
    err = np.abs(r - ref)
    tol = torch.finfo(got.dtype).eps / 2 * np.abs(ref) + c * U * scale
    assert np.all(err <= tol + 1e-37), (what, float(np.max(err - tol)), np.unravel_index(np.argmax(err - tol), err.shape))


@pytest.mark.parametrize("T,H,res,wt,gate", [
    (16500, 264, "bf16", "f32", "channel"), (8300, 1024, "f32", "bf16", "token"), (2900, 1536, "bf16", "bf16", "channel"),
    (2200, 2048, "f32", "f32", "full"), (2100, 4096, "bf16", "bf16", "channel"), (1100, 6400, "f32", "bf16", "token"),
    (600, 16384, "bf16", "bf16", "channel"), (530, 8200, "f32", "f32", "none")])
def test_rows_in_turn(T, H, res, wt, gate):
    import mixture_experts_ffn_int32_amd as hmm
    from mixture_experts_ffn_int32_amd import _lib
    announce("norm rows in turn T=%d H=%d %s %s %s" % (T, H, res, wt, gate))
    g = torch.Generator().manual_seed(23)

    def rnd(*shape):
        return torch.randn(shape, generator=g)
    mag = torch.exp2(torch.randint(-5, 6, (T, 1), generator=g).float())  # rows of their own magnitude
    gv = {"none": None, "token": rnd(T, 1), "channel": rnd(H), "full": rnd(T, H)}[gate]
    v = {"y": (rnd(T, H) * mag.flip(0)).bfloat16(), "residual": (rnd(T, H) * mag).to(TYPES[res]),
         "norm_weight": (1 + 0.3 * rnd(H)).to(TYPES[wt]), "post_weight": (1 + 0.3 * rnd(H)).to(TYPES[wt]),
         "gate": None if gv is None else gv.bfloat16()}
    v = {k: None if t is None else t.cuda().requires_grad_(True) for k, t in v.items()}
    tr, dn = rnd(T, H).to(TYPES[res]).cuda(), rnd(T, H).bfloat16().cuda()
    out, n = hmm.residual_norm(v["y"], v["residual"], v["norm_weight"], post_weight=v["post_weight"], gate=v["gate"], eps=1e-5)
    names = [k for k in v if v[k] is not None]
    grads = torch.autograd.grad((out, n), [v[k] for k in names], (tr, dn))
    f = {k: None if t is None else to_f64(t.detach()) for k, t in v.items()}
    eps = float(np.float32(1e-5))
    _close(out, *block.residual_sum(f["y"], f["residual"], f["post_weight"], f["gate"], 1.0, eps), 256, "residual_out")
    rs = to_f64(out.detach())
    ref = rs * block.rms(rs, eps) * f["norm_weight"]
    _close(n, ref, np.abs(ref), 256, "normed")
    want = block.residual_norm_grads(to_f64(tr), to_f64(dn), f["y"], rs, f["norm_weight"], f["post_weight"], f["gate"], 1.0, eps)
    for k, t in zip(names, grads):
        _close(t, *want["d_" + k], 256 + T, "d_" + k)
    # the C call may write its outputs over its inputs
    kind = {"none": 0, "token": 1, "channel": 2, "full": 3}[gate]
    dt = {"bf16": _lib.HMM_BF16, "f32": _lib.HMM_F32}
    p = _lib.NormProblem(T, H, dt[res], dt[wt], kind, 1e-5, 1.0)
    v = {k: None if t is None else t.detach() for k, t in v.items()}
    a = [None if v[k] is None else ctypes.c_void_p(v[k].data_ptr()) for k in ("y", "residual", "norm_weight", "post_weight", "gate")]
    _lib.check(_lib.load().hmm_residual_norm(ctypes.byref(p), *a, a[1], a[0], None,
                                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    assert torch.equal(v["residual"], out) and torch.equal(v["y"], n)
