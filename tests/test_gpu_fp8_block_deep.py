"""The E4M3 block product over contractions of more than 64 groups of 128 a part: a wave holds 64 groups' block
scales at a time and loads the next 64 on the way.  Each tile size, forward and dx (scales along the other side).

The reference is a 64-bit product of the values that the codes stand for, so it does not use the group structure at
all.  Tolerance, with a the sum of absolute products and b the sum over groups of the largest |x| times the largest
|w| with their scales: y's rounding 2^-8 |y|, 128 2^-13 b for the matrix instruction's alignment (13 bits below the
largest product of a group), and one scaling and one addition a group, at most 8 parts' sums: (groups + 9) 2^-23 a.
The cuts have either sign: the error's 2-norm is held to y's rounding alone.
"""

import pytest
import torch

from _util import announce

pytestmark = pytest.mark.gpu


def _rand(shape, seed, steps):
    """A magnitude of its own for each row's (steps = 1) or each 128 rows' (128) groups of 128 along the second axis."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(shape, generator=g, device="cuda")
    s = torch.randint(-3, 4, ((shape[0] + steps - 1) // steps, (shape[1] + 127) // 128), generator=g, device="cuda").float()
    s = s.repeat_interleave(steps, 0)[:shape[0]].repeat_interleave(128, 1)[:, :shape[1]]
    return (t * torch.exp2(s)).bfloat16()


def _values(codes, descale, steps):
    """64-bit values of codes [n,K], descales [ceil(n/steps),K/128]; and the largest of each row's groups."""
    v = codes.view(torch.float8_e4m3fn).double()
    v = v * descale.double().repeat_interleave(steps, 0)[:v.shape[0]].repeat_interleave(128, 1)
    return v, v.abs().view(v.shape[0], -1, 128).amax(2)


def _check(y, xq, xs, wq, ws):
    (x, xm), (w, wm) = _values(xq, xs, 1), _values(wq, ws, 128)
    ref = torch.matmul(x, w.t().contiguous())
    tol = 2.0 ** -8 * ref.abs() + 128 * 2.0 ** -13 * torch.matmul(xm, wm.t().contiguous())
    tol += (xm.shape[1] + 9) * 2.0 ** -23 * torch.matmul(x.abs(), w.abs().t().contiguous())
    err = (y.double() - ref).abs()
    assert float((err - tol).max()) <= 0, (float((err - tol).max()), float(err.max()))
    assert float(err.norm()) <= 2.0 ** -8 * float(ref.norm())


@pytest.mark.parametrize("T,H,N", [(90, 16640, 272), (130, 8320, 5600), (257, 8448, 8080), (2900, 8320, 2832), (40, 33024, 1040),
                                   (9, 16640, 144), (30, 16640, 272)])
def test_forward(T, H, N):
    import mixture_experts_ffn_int32_amd as hmm
    announce("deep linear_fp8_block %s" % ((T, H, N),))
    x, w = _rand((T, H), 1, 1), _rand((N, H), 2, 128).t().contiguous()
    codes, ds = hmm.quantize_block(w)
    xq, xs = hmm.quantize_rows_block(x)
    y = hmm.linear_fp8_block(x, (codes, ds))
    _check(y, xq, xs, codes, ds)
    z = hmm.matmul_fp8_block(xq, xs, codes, ds)
    assert torch.equal(z, y) if T > 16 else True
    _check(z, xq, xs, codes, ds)


@pytest.mark.parametrize("T,H,N", [(90, 256, 16640), (130, 5632, 8320)])
def test_dx(T, H, N):
    import mixture_experts_ffn_int32_amd as hmm
    announce("deep linear_fp8_block dx %s" % ((T, H, N),))
    w, dy = _rand((H, N), 3, 128), _rand((T, N), 4, 1)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    dx, = torch.autograd.grad(hmm.linear_fp8_block(x, w), x, dy)
    codes, ds = hmm.quantize_block(w)
    gq, gs = hmm.quantize_rows_block(dy)
    _check(dx, gq, gs, codes.t().contiguous(), ds.t().contiguous())
