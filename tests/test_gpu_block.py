"""The operators of a block in a run, as they are used: serving (residual_norm, moe_decode on quantised
weights, linear_fp8_block, residual_norm) and training (rms_norm, linear_fp8_block, hyper_mega_moe,
residual_norm, forward and backward).  Every stage is compared with its float64 reference at the inputs
that it got, with the tolerance of that stage's own tests."""

import numpy as np
import pytest
import torch

from _util import announce, to_f64
from oracle import block

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _f(t):
    return to_f64(t.detach())


def _near(got, ref, scale, c, what):
    err = np.abs(_f(got) - ref)
    assert np.all(err <= torch.finfo(got.dtype).eps / 2 * np.abs(ref) + c * U * scale + 1e-37), (what, err.max())


@pytest.mark.parametrize("T", [1, 7, 40])
def test_serving_block(T):
    import mixture_experts_ffn_int32_amd as hmm
    from test_gpu_decode import _bounds, _layer
    H, I, E, K = 512, 256, 12, 4
    announce("serving block T=%d" % T)
    x, weights, scales, ref = _layer(T, H, I, E, 41, True)
    g = torch.Generator().manual_seed(42)
    stream = (torch.randn((T, H), generator=g) * 2).cuda()
    wpre, wpost = (1 + 0.2 * torch.randn((2, H), generator=g)).cuda()
    wr = (torch.randn((E, H), generator=g) * H ** -0.5).bfloat16().cuda()
    proj = (torch.randn((H, H), generator=g) * H ** -0.5).bfloat16().cuda()
    gate = torch.sigmoid(torch.randn((T, 1), generator=g)).bfloat16().cuda()
    with torch.no_grad():
        a = hmm.linear_fp8_block(x.cuda(), hmm.quantize_block(proj))          # the attention's output projection
        r1, n1 = hmm.residual_norm(a, stream, wpre, eps=1e-5)
        y, ids, w = hmm.moe_decode(n1, *weights, router_weight=wr, top_k=K, **scales)
        r2, n2 = hmm.residual_norm(y, r1, wpre, post_weight=wpost, gate=gate, residual_scale=0.5, eps=1e-5)
    eps = float(np.float32(1e-5))
    v, d = block.quantize_block(proj.float().cpu().numpy())
    xv, xs = block.quantize_rows_block(x.float().numpy())
    aref, big, sabs = block.block_product(xv, xs, v, d)
    # above 16 tokens the E4M3 instruction sums a group's 128 products, each cut at 2^-13 of the
    # group's largest, which `big` holds summed over the groups: 128 2^-13 of it
    cut = 128 * 2.0 ** -13 * big if T > 16 else 0.0
    assert np.all(np.abs(_f(a) - aref) <= 2.0 ** -8 * np.abs(aref) + cut + (H / 128 + 9) * 2.0 ** -23 * sabs)
    want, scale = block.residual_sum(_f(a), _f(stream), None, None, 1.0, eps)
    _near(r1, want, scale, 256, "residual 1")
    want = _f(r1) * block.rms(_f(r1), eps) * _f(wpre)
    _near(n1, want, np.abs(want), 256, "normed 1")
    rid, rw = block.route(_f(n1), _f(wr), K, True)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    want, dev = block.moe(_f(n1), rid, _f(w), *ref, *_bounds(H, I, K))
    assert np.all(np.abs(_f(y) - want) <= 2.0 ** -8 * np.abs(want) + dev)
    want, scale = block.residual_sum(_f(y), _f(r1), _f(wpost), _f(gate), 0.5, eps)
    _near(r2, want, scale, 256, "residual 2")
    want = _f(r2) * block.rms(_f(r2), eps) * _f(wpre)
    _near(n2, want, np.abs(want), 256, "normed 2")


def test_training_block():
    import mixture_experts_ffn_int32_amd as hmm
    T, H, I, E, K = 150, 256, 128, 4, 2
    announce("training block")
    g = torch.Generator().manual_seed(51)

    def rnd(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).bfloat16().cuda().requires_grad_(True)
    x, proj = rnd(T, H), rnd(H, H, std=H ** -0.5)
    up, down = rnd(E, H, 2 * I, std=H ** -0.5), rnd(E, I, H, std=I ** -0.5)
    w0, w1, wp, gate = rnd(H, std=0.3), rnd(H, std=0.3), rnd(H, std=0.3), rnd(H, std=0.3)
    ids = torch.rand((T, E), generator=g).argsort(dim=1)[:, :K].int().cuda()
    tw = torch.softmax(torch.randn((T, K), generator=g), dim=1).cuda().requires_grad_(True)
    eps = float(np.float32(1e-5))
    n0 = hmm.rms_norm(x, w0, eps=1e-5)
    h = hmm.linear_fp8_block(n0, proj)
    y = hmm.hyper_mega_moe(h, ids, tw, up, down)
    r, n = hmm.residual_norm(y, x, w1, post_weight=wp, gate=gate, residual_scale=0.7, eps=1e-5)
    for t in (n0, h, y):
        t.retain_grad()
    tr, dn = rnd(T, H).detach(), rnd(T, H).detach()
    torch.autograd.backward((r, n), (tr, dn))
    torch.cuda.synchronize()
    assert all(t.grad is not None and bool(torch.isfinite(t.grad).all()) for t in (x, proj, up, down, w0, w1, wp, gate, tw))
    s = float(np.float32(0.7))
    want = block.residual_norm_grads(_f(tr), _f(dn), _f(y), _f(r), _f(w1), _f(wp), _f(gate), s, eps)
    c = 256 + T + 512
    for t, k in ((y, "d_y"), (w1, "d_norm_weight"), (wp, "d_post_weight"), (gate, "d_gate")):
        _near(t.grad, *want[k], c, k)
    # the projection's gradients, from the gradient that the experts returned
    v, d = block.quantize_block(_f(proj).astype(np.float32))
    gv, gs = block.quantize_rows_block(_f(h.grad).astype(np.float32))
    ref, big, sabs = block.block_product(gv, gs, v.T, d.T)
    tol = 2.0 ** -8 * np.abs(ref) + 128 * 2.0 ** -13 * big + (H / 128 + 9) * 2.0 ** -23 * sabs
    assert np.all(np.abs(_f(n0.grad) - ref) <= tol)
    ref, sabs = _f(n0).T @ _f(h.grad), np.abs(_f(n0)).T @ np.abs(_f(h.grad))
    assert np.all(np.abs(_f(proj.grad) - ref) <= 2.0 ** -8 * np.abs(ref) + T * 2.0 ** -23 * sabs)
    # x feeds the norm and the residual sum: its gradient is the sum of both, each rounded, added and rounded again
    first = block.residual_norm_grads(np.zeros((T, H)), _f(n0.grad), None, _f(x), _f(w0), None, None, 1.0, eps)
    _near(w0.grad, *first["d_norm_weight"], c, "d_w0")
    a, b = first["d_residual"], want["d_residual"]
    tol = 2.0 ** -8 * (np.abs(a[0]) + np.abs(b[0]) + np.abs(a[0] + b[0])) * (1 + 2.0 ** -8) + c * U * (a[1] + b[1])
    assert np.all(np.abs(_f(x.grad) - (a[0] + b[0])) <= tol)


@pytest.mark.parametrize("T", [3, 15, 31, 64, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_token_stays_alone(T, bad):
    """A NaN or an infinity in one token: its own outputs are not finite, every other token's bits are as without it."""
    import mixture_experts_ffn_int32_amd as hmm
    from test_gpu_decode import _layer
    H, I, E, K = 256, 128, 6, 2
    announce("bad token T=%d %s" % (T, bad))
    x, up, _, _ = _layer(T, H, I, E, 61, False)[:4]
    g = torch.Generator().manual_seed(62)
    x, w = x.cuda(), (torch.randn((H, 400), generator=g) * H ** -0.5).bfloat16().cuda()
    stream, weight = torch.randn((T, H), generator=g).cuda(), torch.ones(H).cuda()
    ids = torch.rand((T, E), generator=g).argsort(dim=1)[:, :K].int().cuda()
    tw = torch.full((T, K), 0.5).cuda()
    ids[T - 2], tw[T - 2] = -1, bad   # a token whose slots are all dropped: zero, whatever its weights

    def run(x):
        with torch.no_grad():
            outs = [hmm.linear_fp8_block(x, hmm.quantize_block(w)), *hmm.residual_norm(x, stream, weight),
                    hmm.matmul_fp8_block(*hmm.quantize_rows_block(x), *hmm.quantize_block(w))]
            if T <= 64:
                outs.append(hmm.moe_decode(x, *up, topk_ids=ids, topk_weights=tw))
                assert not outs[-1][T - 2].any()
        return outs
    want = run(x)
    assert all(bool(torch.isfinite(o).all()) for o in want)
    b = x.clone()
    b[T // 2, 130] = bad
    rest = [t for t in range(T) if t != T // 2]
    for o, r in zip(run(b), want):
        assert torch.equal(o[rest], r[rest])
        if T // 2 != T - 2:
            assert not bool(torch.isfinite(o[T // 2]).all())
