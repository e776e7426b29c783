"""The operators around the experts at the far end of what they accept: arrays of more than 2^32 elements or bytes,
and the widest rows.  Sampled rows against 64-bit products of the same values; tolerances as in the operators' own
tests (an output's rounding, and the float32 arithmetic before it from the length of its chains)."""

import numpy as np
import pytest
import torch

from _util import announce

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


@pytest.fixture(autouse=True)
def _free():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(shape, seed, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=_gen(seed))


def _near(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert got.shape == ref.shape, what
    assert bool((err <= tol).all()), (what, float((err - tol).max()), float(err.max()))


def _sample(T):
    return torch.tensor(sorted({t for t in (0, 1, T // 3, T // 2, T - 2, T - 1)} | {t for t in (
        2 ** 17 - 1, 2 ** 17, 2 ** 18 + 1, 2 ** 19 - 1, 2 ** 19 + 3) if t < T}), device="cuda")


@pytest.mark.parametrize("T,H", [(140001, 16384), (30000003, 80)])
def test_norm(T, H):
    """2.3e9 elements: residual_out, normed and the gradients of sampled rows; the weight's gradient over all rows."""
    import mixture_experts_ffn_int32_amd as hmm
    announce("large norm %s" % ((T, H),))
    y, r = _rand((T, H), 1).requires_grad_(True), _rand((T, H), 2, 2.0).requires_grad_(True)
    w, wp = (1 + _rand((H,), 3, 0.2)).requires_grad_(True), (1 + _rand((H,), 4, 0.2)).requires_grad_(True)
    dn = _rand((T, H), 5)
    out, n = hmm.residual_norm(y, r, w, post_weight=wp, eps=1e-5)
    dy, dr, dw = torch.autograd.grad(n, (y, r, w), dn)
    s, eps = _sample(T), float(np.float32(1e-5))
    with torch.no_grad():
        yf, rf, wf, pf, d = y[s].double(), r[s].double(), w.double(), wp.double(), dn[s].double()

        def rms(v):
            return (v.square().mean(1, keepdim=True) + eps).rsqrt()
        u = yf * rms(yf)
        c = 256 * 2.0 ** -24
        want = rf + u * pf
        _near(out[s], want, 2.0 ** -8 * want.abs() + c * (rf.abs() + (u * pf).abs()), "residual_out")
        x = out[s].double()
        rho = rms(x)
        x = x * rho
        _near(n[s], x * wf, (2.0 ** -8 + c) * (x * wf).abs(), "normed")
        a = d * wf
        m, ma = (a * x).mean(1, keepdim=True), (a * x).abs().mean(1, keepdim=True)
        t, ta = rho * (a - x * m), rho * (a.abs() + x.abs() * ma)
        _near(dr[s], t, 2.0 ** -8 * t.abs() + c * ta, "d_residual")
        b, ba = t * pf, ta * pf.abs()
        v = rms(yf) * (b - u * (b * u).mean(1, keepdim=True))
        va = rms(yf) * (ba + u.abs() * (ba * u.abs()).mean(1, keepdim=True))
        _near(dy[s], v, 2.0 ** -8 * v.abs() + c * va, "d_y")
        total, scale = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 27) // H)
        for i in range(0, T, step):
            x = out[i:i + step].double()
            x = x * rms(x) * dn[i:i + step].double()
            total += x.sum(0)
            scale += x.abs().sum(0)
        # a walker's rows one after another, then at most 4 + 64 sums: rows / 256 of the many rows at the widest
        _near(dw, total, 2.0 ** -8 * total.abs() + (256 + T / 256) * 2.0 ** -24 * scale, "d_norm_weight")


def _values(codes, descale, rows):
    v = codes.view(torch.float8_e4m3fn).double()
    return v * descale.double().repeat_interleave(rows, 0)[:v.shape[0]].repeat_interleave(128, 1)


def _product(y, x, w, what):
    """y of 64-bit values x [T,K], w [N,K]: the matrix instruction's alignment and the sums over groups."""
    ref = torch.matmul(x, w.t().contiguous())
    big = torch.matmul(x.abs().view(x.shape[0], -1, 128).amax(2), w.abs().view(w.shape[0], -1, 128).amax(2).t().contiguous())
    tol = 2.0 ** -8 * ref.abs() + 128 * 2.0 ** -13 * big
    tol += (x.shape[1] / 128 + 9) * U * torch.matmul(x.abs(), w.abs().t().contiguous())
    _near(y, ref, tol, what)
    assert float((y.double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm()), what


@pytest.mark.parametrize("T,H,N", [(600011, 8192, 256), (20000003, 128, 128)])
def test_fp8_rows(T, H, N):
    """More than 2^32 codes of tokens, or twenty million of them; dx as large; dw refused past 4 GiB."""
    import mixture_experts_ffn_int32_amd as hmm
    announce("large fp8 rows %s" % ((T, H, N),))
    x, w = _rand((T, H), 1), _rand((H, N), 2, H ** -0.5)
    codes, ds = hmm.quantize_block(w)
    wv, s = _values(codes, ds, 128), _sample(T)
    xq, xs = hmm.quantize_rows_block(x)
    q1, d1 = hmm.quantize_rows_block(x[s])
    assert torch.equal(xq[s], q1) and torch.equal(xs[s], d1)
    xv = _values(q1, d1, 1)
    _product(hmm.linear_fp8_block(x, (codes, ds))[s], xv, wv, "y")
    _product(hmm.matmul_fp8_block(xq, xs, codes, ds)[s], xv, wv, "y of codes")
    del xq, xs
    x.requires_grad_(True)
    dy = _rand((T, N), 3)
    dx, = torch.autograd.grad(hmm.linear_fp8_block(x, w), x, dy)
    _product(dx[s], _values(*hmm.quantize_rows_block(dy[s]), 1), wv.t().contiguous(), "dx")
    if T * H >= 2 ** 31:
        w.requires_grad_(True)
        with pytest.raises(NotImplementedError, match="4 GiB"):
            torch.autograd.grad(hmm.linear_fp8_block(x, w), w, dy)


@pytest.mark.parametrize("T,H,N", [(5, 65536, 16), (20, 65536, 144), (100, 65536, 272), (3, 128, 262144), (30, 128, 262144),
                                   (300, 256, 262144)])
def test_fp8_widths(T, H, N):
    import mixture_experts_ffn_int32_amd as hmm
    announce("fp8 widths %s" % ((T, H, N),))
    x, w = _rand((T, H), 1), _rand((H, N), 2, H ** -0.5)
    codes, ds = hmm.quantize_block(w)
    xv, wv = _values(*hmm.quantize_rows_block(x), 1), _values(codes, ds, 128)
    _product(hmm.linear_fp8_block(x, (codes, ds)), xv, wv, "y")
    if N % 128 == 0:
        x.requires_grad_(True)
        dy = _rand((T, N), 3)
        dx, = torch.autograd.grad(hmm.linear_fp8_block(x, w), x, dy)
        _product(dx, _values(*hmm.quantize_rows_block(dy), 1), wv.t().contiguous(), "dx")


def test_quantize_block_past_32_bits():
    import mixture_experts_ffn_int32_amd as hmm
    E, H, N = 600, 2048, 4096
    announce("large quantize_block")
    w = _rand((E, H, N), 1)
    codes, ds = hmm.quantize_block(w)
    for e in (0, 1, 255, 256, 512, E - 1):
        c, d = hmm.quantize_block(w[e])
        assert torch.equal(codes[e], c) and torch.equal(ds[e], d)


@pytest.mark.parametrize("T,H,I,E,K,fp8", [
    (9, 7168, 2048, 200, 3, False), (64, 7168, 2048, 200, 3, True),                    # weights past 4 GiB
    (64, 65536, 128, 3, 2, False), (7, 65536, 128, 3, 2, True), (64, 128, 65536, 3, 2, False), (3, 128, 65536, 3, 3, True)])
def test_decode(T, H, I, E, K, fp8):
    import mixture_experts_ffn_int32_amd as hmm
    announce("large moe_decode %s" % ((T, H, I, E, K, fp8),))
    x = _rand((T, H), 1)
    up, down = _rand((E, H, 2 * I), 2, H ** -0.5), _rand((E, I, H), 3, I ** -0.5)
    wr = _rand((E, H), 4, H ** -0.5)
    kw = {}
    if fp8:
        up, kw["up_descale"] = hmm.quantize_block(up)
        down, kw["down_descale"] = hmm.quantize_block(down)
    y, ids, w = hmm.moe_decode(x, up, down, router_weight=wr, top_k=K, **kw)
    logits = torch.matmul(x.double(), wr.double().t().contiguous())
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), order.indices[:, :K])
    _near(w, torch.softmax(order.values[:, :K], 1), (E + 16) * 2.0 ** -24, "weights")
    # chains of H / 2 and I products (bf16, two waves a tile), or of a step's products and the steps
    u = H / 2 + 4 if not fp8 else 128 + H / 128 + 6
    eo = (I + 4 if not fp8 else 256 + I / 128 + 6) + K + 1
    want, dev = torch.zeros((T, H), dtype=torch.float64, device="cuda"), torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.flatten().tolist())):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if fp8:
            W1, W2 = (_values(q[e], kw[n][e], 128).t().contiguous() for q, n in ((up, "up_descale"), (down, "down_descale")))
        else:
            W1, W2 = up[e].double(), down[e].double()
        xe = x[t].double()
        h, ha = torch.matmul(xe, W1), u * U * torch.matmul(xe.abs(), W1.abs())
        g, v = h[:, :I], h[:, I:]
        s = g * torch.sigmoid(g)
        da = 1.1 * ha[:, :I] * v.abs() + s.abs() * ha[:, I:] + (16 * 2.0 ** -24 + 2.0 ** -17) * (s * v).abs()
        we = w[t, k, None].double()
        want[t] += we * torch.matmul(s * v, W2)
        dev[t] += we * torch.matmul(da + eo * U * (s * v).abs(), W2.abs())
    _near(y, want, 2.0 ** -8 * want.abs() + dev, "y")
    assert float((y.double() - want).norm()) <= 2.0 ** -8 * float(want.norm())
