"""moe_decode of one to four tokens, where the workgroup that finishes a column tile last adds the rows up: the
counters that tell it so are cleared in every call, captured ones too, whatever the workspace held."""

import ctypes

import pytest
import torch

from _util import announce
from test_gpu_decode import _layer

pytestmark = pytest.mark.gpu


def _inputs(T, H, I, E, K, fp8):
    x, weights, scales, _ = _layer(T, H, I, E, 71, fp8)
    g = torch.Generator().manual_seed(72)
    ids = torch.rand((2, T, E), generator=g).argsort(dim=2)[:, :, :K].int().contiguous()
    ids[1, 0] = -1           # a token without an expert
    w = torch.rand((T, K), generator=g)
    return x.cuda(), weights, scales, ids.cuda(), w.cuda()


CASES = [(1, 512, 192, 8, 3, False), (3, 1088, 128, 5, 4, False), (4, 512, 256, 16, 8, True), (1, 128, 128, 2, 1, True)]


@pytest.mark.parametrize("T,H,I,E,K,fp8", CASES)
def test_replays(T, H, I, E, K, fp8):
    import mixture_experts_ffn_int32_amd as hmm
    announce("moe_decode replays %s" % ((T, H, I, E, K, fp8),))
    x, weights, scales, ids, w = _inputs(T, H, I, E, K, fp8)
    xs = (x, x.flip(0).contiguous(), -x)

    def call(x, ids):
        return hmm.moe_decode(x, *weights, topk_ids=ids, topk_weights=w, **scales)
    # more experts than tokens, and fewer: the number of workgroups that count differs from replay to replay
    which = [(a, b) for a in range(3) for b in range(2)]
    refs = {k: call(xs[k[0]], ids[k[1]]).clone() for k in which}
    sx, si = x.clone(), ids[0].clone()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(call(sx, si))
    for k in which + which[::-1]:
        sx.copy_(xs[k[0]])
        si.copy_(ids[k[1]])
        for g in graphs:  # one after the other on one stream
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, refs[k]) for o in outs)
        assert torch.equal(call(xs[k[0]], ids[k[1]]), refs[k])


@pytest.mark.parametrize("T,H,I,E,K,fp8", CASES)
@pytest.mark.parametrize("fill", [0, 1, 255])
def test_workspace_contents(T, H, I, E, K, fp8, fill):
    import mixture_experts_ffn_int32_amd as hmm
    from mixture_experts_ffn_int32_amd import _lib
    announce("moe_decode workspace %s %d" % ((T, H, I, E, K, fp8), fill))
    x, weights, scales, ids, w = _inputs(T, H, I, E, K, fp8)
    lib, routed = _lib.load(), [t.clone() for t in ids]  # each from 16 bytes
    prob = _lib.DecodeProblem(T, H, I, E, K, _lib.HMM_FP8_E4M3_BLOCK if fp8 else _lib.HMM_BF16, _lib.HMM_BF16, 0)
    n = ctypes.c_size_t()
    _lib.check(lib.hmm_moe_decode_sizes(ctypes.byref(prob), ctypes.byref(n)))
    work = torch.full((n.value,), fill, dtype=torch.uint8, device="cuda")
    y = torch.full((T + 1, H), 3.0, dtype=torch.bfloat16, device="cuda")

    def p(t):
        return None if t is None else ctypes.c_void_p(t.data_ptr())
    for i in (0, 1, 0):
        want = hmm.moe_decode(x, *weights, topk_ids=ids[i], topk_weights=w, **scales)
        _lib.check(lib.hmm_moe_decode(ctypes.byref(prob), p(x), None, p(routed[i]), p(w), p(weights[0]),
                                      p(scales.get("up_descale")), p(weights[1]), p(scales.get("down_descale")), p(y), p(work),
                                      n.value, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
        torch.cuda.synchronize()
        assert torch.equal(y[:T], want) and bool((y[T] == 3.0).all())
