"""A tangent of forward-mode differentiation is refused, whichever tensor carries it: it would be lost otherwise."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

from _util import announce

pytestmark = pytest.mark.gpu
T, H, I, E, K = 3, 128, 128, 2, 1


def _tensors():
    import mixture_experts_ffn_int32_amd as hmm
    g = torch.Generator().manual_seed(1)

    def rnd(*shape):
        return torch.randn(shape, generator=g).bfloat16().cuda()
    t = {"x": rnd(T, H), "r": rnd(T, H).float(), "w": rnd(H), "wp": rnd(H), "gate": rnd(T, 1), "m": rnd(H, 256),
         "up": rnd(E, H, 2 * I), "down": rnd(E, I, H), "wr": rnd(E, H), "tw": torch.ones(T, K).cuda()}
    t["codes"], t["descale"] = hmm.quantize_block(t["m"])
    t["xq"], t["xs"] = hmm.quantize_rows_block(t["x"])
    (t["upc"], t["upd"]), (t["dnc"], t["dnd"]) = hmm.quantize_block(t["up"]), hmm.quantize_block(t["down"])
    t["ids"] = torch.zeros((T, K), dtype=torch.int32).cuda()
    return t


def _calls():
    import mixture_experts_ffn_int32_amd as hmm
    return {
        "rms_norm": (("x", "w"), lambda t: hmm.rms_norm(t["x"], t["w"])),
        "residual_norm": (("x", "r", "w", "wp", "gate"),
                          lambda t: hmm.residual_norm(t["x"], t["r"], t["w"], post_weight=t["wp"], gate=t["gate"])),
        "linear_fp8_block": (("x", "m"), lambda t: hmm.linear_fp8_block(t["x"], t["m"])),
        "linear_fp8_block of codes": (("x", "descale"), lambda t: hmm.linear_fp8_block(t["x"], (t["codes"], t["descale"]))),
        "matmul_fp8_block": (("xs", "descale"), lambda t: hmm.matmul_fp8_block(t["xq"], t["xs"], t["codes"], t["descale"])),
        "moe_decode": (("x", "wr", "up", "down"), lambda t: hmm.moe_decode(t["x"], t["up"], t["down"], router_weight=t["wr"], top_k=K)),
        "moe_decode E4M3": (("x", "tw", "upd", "dnd"), lambda t: hmm.moe_decode(
            t["x"], t["upc"], t["dnc"], topk_ids=t["ids"], topk_weights=t["tw"], up_descale=t["upd"], down_descale=t["dnd"])),
    }


NAMES = ("rms_norm", "residual_norm", "linear_fp8_block", "linear_fp8_block of codes", "matmul_fp8_block", "moe_decode",
         "moe_decode E4M3")


@pytest.mark.parametrize("name", NAMES)
def test_tangents(name):
    announce("tangents of %s" % name)
    t = _tensors()
    names, call = _calls()[name]
    want = call(t)
    for k in names:
        with fwd.dual_level():
            with pytest.raises(ValueError, match="forward-mode"):
                call(dict(t, **{k: fwd.make_dual(t[k], torch.ones_like(t[k]))}))
            got = call(t)  # the level alone changes nothing
        for a, b in zip(*((o,) if isinstance(o, torch.Tensor) else o for o in (got, want))):
            assert torch.equal(a, b)
