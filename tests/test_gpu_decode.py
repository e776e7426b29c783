"""moe_decode on the GPU against the float64 reference (oracle/block.py).

ids are compared exactly: the logits are sums of exact products in 64 bits.  y is off by its
rounding (2^-8 of it) and by the float32 arithmetic before it, bounded per stage:
* the up-projection's sums: a chain of at most H / 8 + 8 additions (every 8th step of 32 in
  one wave, the matrix instruction's 32 products in turn, 8 waves), each off by at most
  2^-23 of the absolute sum, and for E4M3 one scaling per group more;
* a: silu's exponential, reciprocal and products (16 2^-24), kept as two bf16 (2^-17);
* the down-projection's sums as the first, and K + 1 weighted additions.
The routing weights: exponential, sum over E and division, 2 + E in a chain of 2^-24.
"""

import numpy as np
import pytest
import torch

from _util import announce, to_f64
from oracle import block

pytestmark = pytest.mark.gpu


def _bounds(H, I, K):
    u = 2.0 ** -23
    return (H / 8 + H / 128 + 16) * u, 16 * 2.0 ** -24 + 2.0 ** -17, (I / 8 + I / 128 + 16 + K + 1) * u


def _layer(T, H, I, E, seed, fp8):
    import mixture_experts_ffn_int32_amd as hmm
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g).bfloat16()
    up = (torch.randn((E, H, 2 * I), generator=g) * H ** -0.5).bfloat16()
    down = (torch.randn((E, I, H), generator=g) * I ** -0.5).bfloat16()
    if not fp8:
        uf, df = up.float().numpy(), down.float().numpy()
        ref = (lambda e: uf[_in(e, E)].astype(np.float64), lambda e: df[_in(e, E)].astype(np.float64))
        return x, (up.cuda(), down.cuda()), {}, ref
    (uc, ud), (dc, dd) = hmm.quantize_block(up.cuda()), hmm.quantize_block(down.cuda())

    def values(c, d):
        c, d = c.cpu().numpy(), d.cpu().numpy().astype(np.float64)

        def of(e):
            s = np.repeat(np.repeat(d[_in(e, E)], 128, axis=0), 128, axis=1)
            return (block.e4m3_values(c[e]) * s).T
        return of
    return x, (uc, dc), {"up_descale": ud, "down_descale": dd}, (values(uc, ud), values(dc, dd))


def _in(e, E):
    if not 0 <= e < E:
        raise IndexError(e)
    return e


def _check(y, x, ids, w, ref, H, I):
    want, dev = block.moe(x.float().numpy().astype(np.float64), ids, w, *ref, *_bounds(H, I, ids.shape[1]))
    err = np.abs(to_f64(y) - want)
    tol = 2.0 ** -8 * np.abs(want) + dev
    assert np.all(err <= tol + 1e-37), (float(np.max(err - tol)), float(np.max(err)))


SHAPES = [  # T, H, I, E, K, fp8
    (1, 64, 64, 1, 1, False), (1, 512, 128, 4, 2, False), (4, 512, 128, 4, 2, False), (3, 192, 320, 5, 3, False),
    (16, 256, 192, 33, 8, False), (17, 448, 64, 7, 2, False), (32, 320, 128, 3, 3, False), (33, 128, 192, 6, 1, False),
    (64, 256, 128, 4, 4, False), (64, 576, 64, 70, 8, False), (2, 128, 64, 1024, 16, False),
    # wide tiles of both projections, with a last column tile of 64, for one and for two row tiles
    (16, 1088, 512, 128, 8, False), (64, 1088, 512, 128, 8, False), (64, 1344, 640, 120, 16, False),
    (1, 128, 128, 1, 1, True), (5, 512, 128, 4, 2, True), (16, 256, 384, 9, 4, True), (23, 640, 128, 5, 3, True),
    (64, 384, 256, 6, 6, True), (48, 256, 128, 40, 2, True),
]


@pytest.mark.parametrize("T,H,I,E,K,fp8", SHAPES)
def test_given_routing(T, H, I, E, K, fp8):
    import mixture_experts_ffn_int32_amd as hmm
    announce("moe_decode %s" % ((T, H, I, E, K, fp8),))
    x, weights, scales, ref = _layer(T, H, I, E, 3, fp8)
    g = torch.Generator().manual_seed(4)
    ids = torch.rand((T, E), generator=g).argsort(dim=1)[:, :K].int()
    w = torch.softmax(torch.randn((T, K), generator=g), dim=1)
    y = hmm.moe_decode(x.cuda(), *weights, topk_ids=ids.cuda(), topk_weights=w.cuda(), **scales)
    torch.cuda.synchronize()
    _check(y, x, ids.numpy(), w.numpy().astype(np.float64), ref, H, I)


@pytest.mark.parametrize("T,H,I,E,fp8", [(64, 192, 128, 40, False), (50, 256, 128, 40, True), (64, 1088, 512, 128, False)])
def test_crowded_expert(T, H, I, E, fp8):
    """Many experts, so that few rows each are expected, and all tokens go to two of them."""
    import mixture_experts_ffn_int32_amd as hmm
    announce("moe_decode crowded expert %s" % ((T, H, I, E, fp8),))
    x, weights, scales, ref = _layer(T, H, I, E, 31, fp8)
    g = torch.Generator().manual_seed(32)
    ids = torch.tensor([[E - 1, 3]]).repeat(T, 1).int()
    ids[1] = torch.tensor([5, 3])
    w = torch.rand((T, 2), generator=g)
    y = hmm.moe_decode(x.cuda(), *weights, topk_ids=ids.cuda(), topk_weights=w.cuda(), **scales)
    _check(y, x, ids.numpy(), w.numpy(), ref, H, I)


@pytest.mark.parametrize("fp8", [False, True])
def test_repeated_and_invalid_ids(fp8):
    """A token that names an expert twice, ids out of range (dropped), a token with none, and none at all."""
    import mixture_experts_ffn_int32_amd as hmm
    T, H, I, E = 6, 256, 128, 4
    announce("moe_decode repeated and invalid ids fp8=%s" % fp8)
    x, weights, scales, ref = _layer(T, H, I, E, 5, fp8)
    ids = torch.tensor([[1, 1, 2], [3, -1, 3], [-1, -1, -1], [4, 1000000, 0], [2, 2, 2], [0, 1, -7]], dtype=torch.int32)
    w = torch.tensor([[0.5, 0.25, 0.25], [1.0, 9.0, -0.5], [1, 1, 1], [3, 3, 0.5], [0.1, 0.2, 0.3], [0.0, 1.0, 5.0]])
    y = hmm.moe_decode(x.cuda(), *weights, topk_ids=ids.cuda(), topk_weights=w.cuda(), **scales)
    _check(y, x, ids.numpy(), w.numpy().astype(np.float64), ref, H, I)
    assert not y[2].any()
    far = ids.long()
    far[far == -1] = (1 << 32) + 1  # 64-bit ids that a cut to 32 bits would make valid
    assert torch.equal(hmm.moe_decode(x.cuda(), *weights, topk_ids=far.cuda(), topk_weights=w.cuda(), **scales), y)
    none = hmm.moe_decode(x.cuda(), *weights, topk_ids=torch.full_like(ids, -1).cuda(), topk_weights=w.cuda(), **scales)
    assert not none.any()


@pytest.mark.parametrize("T,H,I,E,K,fp8,renorm,dt", [
    (1, 512, 128, 4, 2, False, True, "bf16"), (5, 1152, 64, 32, 8, False, False, "bf16"), (64, 128, 64, 129, 8, False, True, "f32"),
    (17, 256, 128, 1024, 16, True, False, "bf16"), (2, 4160, 64, 3, 3, False, False, "f32"), (9, 64, 64, 1, 1, False, True, "bf16")])
def test_router(T, H, I, E, K, fp8, renorm, dt):
    import mixture_experts_ffn_int32_amd as hmm
    announce("moe_decode router %s" % ((T, H, I, E, K, fp8, renorm, dt),))
    g = torch.Generator().manual_seed(8)
    if E == 1024:  # the weights of a thousand experts would be large: one tiny set, expanded
        x, weights, scales, ref = _layer(T, H, I, 1, 7, fp8)
        weights = tuple(t.expand(E, -1, -1).contiguous() for t in weights)
        scales = {k: t.expand(E, -1, -1).contiguous() for k, t in scales.items()}
        ref = tuple((lambda f: lambda e: f(0))(f) for f in ref)
    else:
        x, weights, scales, ref = _layer(T, H, I, E, 7, fp8)
    wr = (torch.randn((E, H), generator=g) * H ** -0.5).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    y, ids, w = hmm.moe_decode(x.cuda(), *weights, router_weight=wr.cuda(), top_k=K, renormalize=renorm, **scales)
    xf = x.float().numpy().astype(np.float64)
    rid, rw = block.route(xf, wr.float().numpy().astype(np.float64), K, renorm)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=(E + 16) * 2.0 ** -24, atol=1e-37)
    _check(y, x, rid, w.cpu().numpy().astype(np.float64), ref, H, I)


def test_router_ties_and_nan():
    """Equal logits go to the lower expert, whatever the order of the sums; a NaN logit ranks last."""
    import mixture_experts_ffn_int32_amd as hmm
    T, H, I, E, K = 3, 1024, 64, 130, 6
    x, weights, _, _ = _layer(T, H, I, 1, 1, False)
    weights = tuple(t.expand(E, -1, -1).contiguous() for t in weights)
    x[1] = 0.0  # every logit equal
    g = torch.Generator().manual_seed(2)
    row = torch.randn((1, H), generator=g).bfloat16()
    wr = row.repeat(E, 1)
    wr[::2] = -row
    y, ids, w = hmm.moe_decode(x.cuda(), *weights, router_weight=wr.cuda(), top_k=K)
    rid, _ = block.route(x.float().numpy().astype(np.float64), wr.float().numpy().astype(np.float64), K, True)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    assert ids[1].tolist() == list(range(K))
    wr[3:] = float("nan")
    y, ids, w = hmm.moe_decode(x.cuda(), *weights, router_weight=wr.cuda(), top_k=K)
    assert all(sorted(r[:3]) == [0, 1, 2] and r[3:] == [3, 4, 5] for r in ids.tolist())


def test_views_streams_workspaces_and_graph():
    """Rows of a larger batch, another stream, two calls side by side, and a captured call replayed on new routing."""
    import mixture_experts_ffn_int32_amd as hmm
    T, H, I, E, K = 12, 512, 192, 8, 3
    x, weights, _, _ = _layer(T, H, I, E, 21, False)
    x = x.cuda()
    g = torch.Generator().manual_seed(22)
    wr = torch.randn((E, H), generator=g).bfloat16().cuda()

    def call(x):
        return hmm.moe_decode(x, *weights, router_weight=wr, top_k=K)
    y, ids, w = call(x)
    for a, b in ((0, 5), (5, 6), (1, 12)):  # a token's result does not depend on its neighbours
        ys, i2, w2 = call(x[a:b])
        assert torch.equal(ys, y[a:b]) and torch.equal(i2, ids[a:b]) and torch.equal(w2, w[a:b])
        part = hmm.moe_decode(x[a:b], *weights, topk_ids=ids[a:b], topk_weights=w[a:b])  # views off 16 bytes
        assert torch.equal(part, y[a:b])
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(call(x)[0])
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o in outs)
    x2 = x.flip(0).contiguous()
    refs = [tuple(t.clone() for t in call(v)) for v in (x, x2)]
    static = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(static)
    for which in (1, 0, 1):
        static.copy_((x, x2)[which])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, refs[which]))
        call(x2)
        torch.cuda.synchronize()


def test_workspace_contents_do_not_matter():
    """The workspace may hold anything (all ones here), and rows behind the last token stay as they were."""
    import ctypes
    import mixture_experts_ffn_int32_amd as hmm
    from mixture_experts_ffn_int32_amd import _lib
    T, H, I, E, K = 5, 192, 128, 6, 2
    x, (up, down), _, _ = _layer(T, H, I, E, 31, False)
    g = torch.Generator().manual_seed(3)
    wr = torch.randn((E, H), generator=g).bfloat16().cuda()
    x = x.cuda()
    want = hmm.moe_decode(x, up, down, router_weight=wr, top_k=K)
    lib = _lib.load()
    prob = _lib.DecodeProblem(T, H, I, E, K, _lib.HMM_BF16, _lib.HMM_BF16, _lib.HMM_DECODE_RENORMALIZE)
    n = ctypes.c_size_t()
    _lib.check(lib.hmm_moe_decode_sizes(ctypes.byref(prob), ctypes.byref(n)))
    work = torch.full((n.value + 64,), 255, dtype=torch.uint8, device="cuda")
    y = torch.full((T + 1, H), 3.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T + 1, K), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, K), -9.0, device="cuda")

    def p(t):
        return ctypes.c_void_p(t.data_ptr())
    for _ in range(2):
        _lib.check(lib.hmm_moe_decode(ctypes.byref(prob), p(x), p(wr), p(ids), p(w), p(up), None, p(down), None, p(y), p(work),
                                      n.value, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
        torch.cuda.synchronize()
        assert torch.equal(y[:T], want[0]) and torch.equal(ids[:T], want[1]) and torch.equal(w[:T], want[2])
        assert bool((y[T] == 3.0).all()) and bool((ids[T] == -9).all()) and bool((w[T] == -9.0).all())
        assert bool((work[n.value:] == 255).all())


def test_no_tokens():
    import mixture_experts_ffn_int32_amd as hmm
    x, weights, _, _ = _layer(0, 128, 64, 2, 1, False)
    y, ids, w = hmm.moe_decode(x.cuda(), *weights, router_weight=torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda"), top_k=2)
    assert y.shape == (0, 128) and ids.shape == w.shape == (0, 2)
