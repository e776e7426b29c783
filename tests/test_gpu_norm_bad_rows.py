"""residual_norm and rms_norm of rows that hold an infinity, a NaN or squares past float32: what the row gives is
fixed, and every other row keeps its bits."""

import pytest
import torch

from _util import announce

pytestmark = pytest.mark.gpu


def test_infinities_and_large_rows():
    """What a row that is not finite gives: a NaN makes the whole row NaN; an infinity of the stream makes its own
    column NaN and the others zero, as does a sum of squares past float32 of a finite row (without the NaN); other
    rows keep their bits."""
    import mixture_experts_ffn_int32_amd as hmm
    T, H = 7, 520
    announce("norm infinities")
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn((T, H), generator=g).cuda(), torch.rand(H, generator=g).cuda() + 0.5
    y = torch.randn((T, H), generator=g).bfloat16().cuda()
    clean, ref = hmm.rms_norm(x, w), hmm.residual_norm(y, x, w, post_weight=w)
    x[1, 17], x[2, 18], x[4, 19] = float("inf"), float("-inf"), float("nan")
    x[5] = x[5].sign() * 1e19  # the squares' sum, 5e40, is infinite in float32
    n = hmm.rms_norm(x, w)
    rest = [0, 3, 6]
    assert torch.equal(n[rest], clean[rest])
    for t, c in ((1, 17), (2, 18)):
        assert bool(torch.isnan(n[t, c])) and not n[t, :c].any() and not n[t, c + 1:].any()
    assert bool(torch.isnan(n[4]).all()) and not n[5].any()
    x = torch.where(torch.isfinite(x) & (x.abs() < 1e18), x, torch.zeros_like(x))
    want = hmm.residual_norm(y, x, w, post_weight=w)
    y[3, 40] = float("inf")  # of the block: the post-norm turns its row's other columns into zeros, its own into NaN
    y[6, 41] = float("nan")
    r, n = hmm.residual_norm(y, x, w, post_weight=w)
    rest = [0, 1, 2, 4, 5]
    assert torch.equal(r[rest], want[0][rest]) and torch.equal(n[rest], want[1][rest])
    assert bool(torch.isnan(r[3, 40])) and torch.equal(r[3, :40], x[3, :40]) and torch.equal(r[3, 41:], x[3, 41:])
    assert bool(torch.isnan(r[6]).all()) and bool(torch.isnan(n[[3, 6]]).all())
    assert bool(torch.isfinite(ref[1]).all())
