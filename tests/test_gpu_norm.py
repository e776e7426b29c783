"""residual_norm and rms_norm on the GPU against the float64 reference (oracle/block.py).

Tolerances: an output of type t is off by its rounding, eps(t) / 2 of its value, and by
the float32 arithmetic before it: at most C roundings of 2^-24 of the sum of its absolute
terms.  A row sum has at most 16 terms per thread, 6 + 16 steps of tree and a few more
operations, and a gradient chains two of them: C = 256.  A column sum over T rows has
T / 512 + 1 rows in one walker, then at most 256 partial rows in one chain: C = 256 + T + 512.
The reference's n and gradients are taken at the stored residual_out, as the definition says.
"""

import numpy as np
import pytest
import torch

from _util import announce, to_f64
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _half_ulp(dtype):
    return torch.finfo(dtype).eps / 2


def _inputs(T, H, res, wt, gate, post, seed):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape):
        return torch.randn(shape, generator=g)
    v = {"y": rnd(T, H).bfloat16(), "residual": (rnd(T, H) * 3).to(res), "norm_weight": (1 + 0.3 * rnd(H)).to(wt),
         "post_weight": (1 + 0.3 * rnd(H)).to(wt) if post else None,
         "gate": {"none": None, "token": rnd(T, 1), "channel": rnd(H), "full": rnd(T, H)}[gate]}
    if v["gate"] is not None:
        v["gate"] = v["gate"].bfloat16()
    if T > 2:
        v["y"][1] = 0          # a block that gave nothing for a token
        v["residual"][2] *= 1e4  # a row far larger than its neighbours
    v = {k: None if t is None else t.cuda() for k, t in v.items()}
    v["tr"], v["dn"] = rnd(T, H).to(res).cuda(), rnd(T, H).bfloat16().cuda()
    return v


def _f64(t):
    return None if t is None else to_f64(t.detach())


def _close(got, ref, scale, c, what):
    r = to_f64(got.detach())
    tol = _half_ulp(got.dtype) * np.abs(ref) + c * U * scale
    err = np.abs(r - ref)
    assert r.shape == ref.shape, what
    assert np.all(err <= tol + 1e-37), (what, float(np.max(err - tol)), float(np.max(err)))


NAMES = ("y", "residual", "norm_weight", "post_weight", "gate")
CASES = [
    (1, 8, "bf16", "bf16", "none", True), (1, 7168, "bf16", "bf16", "token", True), (3, 512, "f32", "f32", "channel", True),
    (5, 520, "bf16", "f32", "full", True), (37, 1024, "bf16", "bf16", "channel", False), (7, 1032, "f32", "bf16", "token", True),
    (130, 2048, "bf16", "bf16", "full", False), (1300, 264, "f32", "f32", "channel", True), (5, 4096, "bf16", "bf16", "none", False),
    (700, 4104, "f32", "f32", "token", False), (3, 8192, "bf16", "bf16", "channel", True), (4, 8200, "f32", "f32", "full", True),
    (2, 16384, "bf16", "bf16", "channel", True), (2500, 96, "bf16", "bf16", "token", True),
    (6, 1536, "bf16", "f32", "full", True), (900, 1544, "f32", "bf16", "channel", True), (2100, 504, "bf16", "bf16", "channel", True),
    (2400, 7176, "bf16", "bf16", "token", True),  # outputs past the L2 caches
]


@pytest.mark.parametrize("T,H,res,wt,gate,post", CASES)
def test_forward_and_gradients(T, H, res, wt, gate, post):
    import mixture_experts_ffn_int32_amd as hmm
    types = {"bf16": torch.bfloat16, "f32": torch.float32}
    announce("residual_norm T=%d H=%d %s %s gate=%s post=%s" % (T, H, res, wt, gate, post))
    v = _inputs(T, H, types[res], types[wt], gate, post, 11)
    names = [k for k in NAMES if v[k] is not None]
    for k in names:
        v[k].requires_grad_(True)
    scale, eps = 0.6, 1e-5
    out, n = hmm.residual_norm(v["y"], v["residual"], v["norm_weight"], post_weight=v["post_weight"], gate=v["gate"],
                               residual_scale=scale, eps=eps)
    grads = torch.autograd.grad((out, n), [v[k] for k in names], (v["tr"], v["dn"]))
    torch.cuda.synchronize()
    assert out.dtype == types[res] and n.dtype == torch.bfloat16
    f = {k: _f64(t) for k, t in v.items()}
    scale, eps = float(np.float32(scale)), float(np.float32(eps))
    ref, absr = block.residual_sum(f["y"], f["residual"], f["post_weight"], f["gate"], scale, eps)
    _close(out, ref, absr, 256, "residual_out")
    rs = _f64(out)
    nref = rs * block.rms(rs, eps) * f["norm_weight"]
    _close(n, nref, np.abs(nref), 256, "normed")
    want = block.residual_norm_grads(f["tr"], f["dn"], f["y"], rs, f["norm_weight"], f["post_weight"], f["gate"], scale, eps)
    for k, g in zip(names, grads):
        assert g.dtype == v[k].dtype
        _close(g, want["d_" + k][0], want["d_" + k][1], 256 + T + 512, "d_" + k)


@pytest.mark.parametrize("T,H,dt", [(1, 64, torch.bfloat16), (9, 3000, torch.float32), (600, 1024, torch.bfloat16)])
def test_rms_norm(T, H, dt):
    import mixture_experts_ffn_int32_amd as hmm
    announce("rms_norm T=%d H=%d %s" % (T, H, dt))
    v = _inputs(T, H, dt, dt, "none", False, 5)
    x, w = v["residual"].requires_grad_(True), v["norm_weight"].requires_grad_(True)
    n = hmm.rms_norm(x, w, eps=1e-5)
    dx, dw = torch.autograd.grad(n, (x, w), v["dn"])
    xf, wf, eps = _f64(x), _f64(w), float(np.float32(1e-5))
    ref = xf * block.rms(xf, eps) * wf
    _close(n, ref, np.abs(ref), 256, "normed")
    want = block.residual_norm_grads(np.zeros_like(xf), _f64(v["dn"]), None, xf, wf, None, None, 1.0, eps)
    _close(dx, *want["d_residual"], 256, "dx")
    _close(dw, *want["d_norm_weight"], 256 + T + 512, "dw")


def test_one_output_used_and_strided_inputs():
    """Only one of the two outputs has a gradient; inputs that are views with other strides."""
    import mixture_experts_ffn_int32_amd as hmm
    T, H = 33, 256
    v = _inputs(T, H, torch.bfloat16, torch.bfloat16, "channel", True, 7)
    wide = torch.cat([v["y"], v["y"]], dim=1)
    y = wide[:, :H]                              # row pitch 2H
    r = v["residual"].t().contiguous().t()       # column major
    out, n = hmm.residual_norm(y, r, v["norm_weight"], post_weight=v["post_weight"], gate=v["gate"])
    o2, n2 = hmm.residual_norm(v["y"], v["residual"], v["norm_weight"], post_weight=v["post_weight"], gate=v["gate"])
    assert torch.equal(out, o2) and torch.equal(n, n2)
    for which in (0, 1):
        leaves = [t.detach().clone().requires_grad_(True) for t in (v["y"], v["residual"], v["norm_weight"])]
        o = hmm.residual_norm(*leaves, post_weight=v["post_weight"], gate=v["gate"])
        got = torch.autograd.grad(o[which], leaves, (v["tr"], v["dn"])[which], allow_unused=True)
        zero = torch.zeros_like(v["tr"])
        leaves2 = [t.detach().clone().requires_grad_(True) for t in leaves]
        o = hmm.residual_norm(*leaves2, post_weight=v["post_weight"], gate=v["gate"])
        want = torch.autograd.grad(o, leaves2, (v["tr"], zero) if which == 0 else (zero, v["dn"]))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,H,res", [(1100, 7168, torch.bfloat16), (4500, 264, torch.float32), (9, 16384, torch.float32)])
def test_outputs_over_the_inputs(T, H, res):
    """residual_out on residual and normed on y, as the C call allows, with more rows than are taken at once."""
    import ctypes
    import mixture_experts_ffn_int32_amd as hmm
    from mixture_experts_ffn_int32_amd import _lib
    announce("norm in place %s" % ((T, H, res),))
    v = _inputs(T, H, res, torch.bfloat16, "channel", True, 19)
    out, n = hmm.residual_norm(v["y"], v["residual"], v["norm_weight"], post_weight=v["post_weight"], gate=v["gate"], eps=1e-5)
    p = _lib.NormProblem(T, H, _lib.HMM_F32 if res == torch.float32 else _lib.HMM_BF16, _lib.HMM_BF16, _lib.HMM_GATE_CHANNEL,
                         1e-5, 1.0)
    a = [ctypes.c_void_p(v[k].data_ptr()) for k in ("y", "residual", "norm_weight", "post_weight", "gate")]
    _lib.check(_lib.load().hmm_residual_norm(ctypes.byref(p), *a, a[1], a[0], None,
                                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    assert torch.equal(v["residual"], out) and torch.equal(v["y"], n)


def test_no_rows():
    import mixture_experts_ffn_int32_amd as hmm
    v = _inputs(0, 64, torch.bfloat16, torch.bfloat16, "channel", True, 7)
    leaves = [v[k].requires_grad_(True) for k in NAMES]
    out, n = hmm.residual_norm(v["y"], v["residual"], v["norm_weight"], post_weight=v["post_weight"], gate=v["gate"])
    assert out.shape == n.shape == (0, 64)
    grads = torch.autograd.grad((out, n), leaves, (v["tr"], v["dn"]))
    assert all(g.shape == t.shape and not g.any() for g, t in zip(grads, leaves))


def test_repeats_streams_and_graph():
    """The same bits on every call, on another stream, and from a captured forward and backward replayed on new inputs."""
    import mixture_experts_ffn_int32_amd as hmm
    T, H = 600, 1032
    ins = [_inputs(T, H, torch.bfloat16, torch.bfloat16, "channel", True, s) for s in (1, 2)]

    def step(v):
        leaves = [v[k].detach().requires_grad_(True) for k in NAMES]
        out, n = hmm.residual_norm(leaves[0], leaves[1], leaves[2], post_weight=leaves[3], gate=leaves[4])
        return (out, n) + torch.autograd.grad((out, n), leaves, (v["tr"], v["dn"]))
    ref = [tuple(t.detach().clone() for t in step(v)) for v in ins]
    assert all(torch.equal(a, b) for a, b in zip(step(ins[0]), ref[0]))
    static = {k: t.clone() for k, t in ins[0].items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step(static)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(other, ref[0]))
    del other
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(static)
    for which in (1, 0, 1):
        for k, t in ins[which].items():
            static[k].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref[which]))
        step(ins[1 - which])
        torch.cuda.synchronize()
