"""A gradient asked of a call that has none is refused, whichever tensor asks for it, and the call runs under no_grad."""

import pytest
import torch

from _util import announce

pytestmark = pytest.mark.gpu
T, H, I, E, K = 3, 128, 128, 2, 1


def _tensors():
    import mixture_experts_ffn_int32_amd as hmm
    g = torch.Generator().manual_seed(1)

    def rnd(*shape):
        return torch.randn(shape, generator=g).bfloat16().cuda()
    t = {"x": rnd(T, H), "m": rnd(H, 256), "up": rnd(E, H, 2 * I), "down": rnd(E, I, H), "wr": rnd(E, H),
         "tw": torch.ones(T, K).cuda()}
    t["codes"], t["descale"] = hmm.quantize_block(t["m"])
    t["xq"], t["xs"] = hmm.quantize_rows_block(t["x"])
    (t["upc"], t["upd"]), (t["dnc"], t["dnd"]) = hmm.quantize_block(t["up"]), hmm.quantize_block(t["down"])
    t["ids"] = torch.zeros((T, K), dtype=torch.int32).cuda()
    return t


def _calls():
    import mixture_experts_ffn_int32_amd as hmm
    return {
        "linear_fp8_block of codes": (("x", "descale"), lambda t: hmm.linear_fp8_block(t["x"], (t["codes"], t["descale"]))),
        "matmul_fp8_block": (("xs", "descale"), lambda t: hmm.matmul_fp8_block(t["xq"], t["xs"], t["codes"], t["descale"])),
        "moe_decode": (("x", "wr", "up", "down"), lambda t: hmm.moe_decode(t["x"], t["up"], t["down"], router_weight=t["wr"], top_k=K)),
        "moe_decode E4M3": (("x", "tw", "upd", "dnd"), lambda t: hmm.moe_decode(
            t["x"], t["upc"], t["dnc"], topk_ids=t["ids"], topk_weights=t["tw"], up_descale=t["upd"], down_descale=t["dnd"])),
    }


NAMES = ("linear_fp8_block of codes", "matmul_fp8_block", "moe_decode", "moe_decode E4M3")


@pytest.mark.parametrize("name", NAMES)
def test_gradients(name):
    announce("gradients of %s" % name)
    t = _tensors()
    names, call = _calls()[name]
    want = call(t)
    for k in names:
        d = dict(t, **{k: t[k].clone().requires_grad_(True)})
        with pytest.raises(ValueError, match="gradient"):
            call(d)
        with torch.no_grad():
            got = call(d)
        for a, b in zip(*((o,) if isinstance(o, torch.Tensor) else o for o in (got, want))):
            assert torch.equal(a, b)
