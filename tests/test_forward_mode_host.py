"""Forward-mode tangents are refused before anything else is looked at (no GPU is touched): the operators
around the experts have no forward-mode derivative, and a dual tensor does not require a gradient."""

import pytest
import torch
import torch.autograd.forward_ad as fwd

import mixture_experts_ffn_int32_amd as hmm


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


CALLS = {
    "rms_norm": lambda d: hmm.rms_norm(d(_bf16(2, 128)), _bf16(128)),
    "residual_norm": lambda d: hmm.residual_norm(_bf16(2, 128), d(_bf16(2, 128)), _bf16(128)),
    "linear_fp8_block": lambda d: hmm.linear_fp8_block(d(_bf16(2, 128)), _bf16(128, 128)),
    "linear_fp8_block of codes": lambda d: hmm.linear_fp8_block(
        d(_bf16(2, 128)), (torch.zeros((16, 128), dtype=torch.uint8), torch.ones(1, 1))),
    "quantize_block": lambda d: hmm.quantize_block(d(_bf16(128, 128))),
    "quantize_rows_block": lambda d: hmm.quantize_rows_block(d(_bf16(2, 128))),
    "moe_decode": lambda d: hmm.moe_decode(d(_bf16(2, 128)), _bf16(1, 128, 128), _bf16(1, 64, 128),
                                           router_weight=_bf16(1, 128), top_k=1),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_tangents_are_refused(name):
    with fwd.dual_level():
        with pytest.raises(ValueError, match="forward-mode"):
            CALLS[name](lambda t: fwd.make_dual(t, torch.ones_like(t)))
        with pytest.raises(ValueError, match="HIP device"):  # inside a dual level, without a tangent
            CALLS[name](lambda t: t)
    with pytest.raises(ValueError, match="HIP device"):
        CALLS[name](lambda t: t)
