"""Refusals of the norms' entry points, all on the host (no GPU is touched)."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_int32_amd as hmm
from mixture_experts_ffn_int32_amd import _lib


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _prob(**kw):
    d = dict(T=4, H=64, residual_dtype=_lib.HMM_BF16, weight_dtype=_lib.HMM_BF16, gate_kind=_lib.HMM_GATE_NONE,
             eps=1e-6, residual_scale=1.0)
    d.update(kw)
    return _lib.NormProblem(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), _lib.HMM_ERR_BAD_SHAPE), (dict(T=1 << 31), _lib.HMM_ERR_BAD_SHAPE), (dict(H=0), _lib.HMM_ERR_BAD_SHAPE),
    (dict(H=60), _lib.HMM_ERR_BAD_SHAPE), (dict(H=16392), _lib.HMM_ERR_BAD_SHAPE), (dict(residual_dtype=2), _lib.HMM_ERR_BAD_DTYPE),
    (dict(weight_dtype=-1), _lib.HMM_ERR_BAD_DTYPE), (dict(gate_kind=4), _lib.HMM_ERR_BAD_SHAPE), (dict(eps=0.0), _lib.HMM_ERR_BAD_SHAPE),
    (dict(eps=float("nan")), _lib.HMM_ERR_BAD_SHAPE), (dict(eps=float("inf")), _lib.HMM_ERR_BAD_SHAPE),
    (dict(residual_scale=float("inf")), _lib.HMM_ERR_BAD_SHAPE), (dict(residual_scale=float("nan")), _lib.HMM_ERR_BAD_SHAPE),
    (dict(), _lib.HMM_OK), (dict(H=16384, gate_kind=3), _lib.HMM_OK)])
def test_problem(lib, kw, status):
    n = ctypes.c_size_t()
    assert lib.hmm_residual_norm_backward_sizes(ctypes.byref(_prob(**kw)), ctypes.byref(n)) == status


def test_pointers(lib):
    z, ok, bad = ctypes.c_void_p(0), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)

    def fwd(p, y=ok, r=ok, w=ok, wp=z, g=z, out=ok, n=ok, rstd=z):
        return lib.hmm_residual_norm(ctypes.byref(p), y, r, w, wp, g, out, n, rstd, z)
    for kw in (dict(r=z), dict(w=z), dict(out=z), dict(n=z)):
        assert fwd(_prob(), **kw) == _lib.HMM_ERR_NULL_POINTER, kw
    for k in ("y", "r", "w", "wp", "out", "n", "rstd"):
        assert fwd(_prob(), **{k: bad}) == _lib.HMM_ERR_MISALIGNED, k
    assert fwd(_prob(gate_kind=1)) == _lib.HMM_ERR_NULL_POINTER
    # the norm alone takes neither a post weight, nor a residual output, nor a gate
    assert fwd(_prob(), y=z) == _lib.HMM_ERR_BAD_SHAPE
    assert fwd(_prob(), y=z, out=z, wp=ok) == _lib.HMM_ERR_BAD_SHAPE
    assert fwd(_prob(gate_kind=2), y=z, out=z, g=ok) == _lib.HMM_ERR_BAD_SHAPE

    def bwd(p, ws=ok, nbytes=1 << 30, y=ok, dy=ok, wp=z, dwp=z, g=z, dg=z, rstd=ok):
        return lib.hmm_residual_norm_backward(ctypes.byref(p), ok, ok, y, ok, ok, wp, g, rstd, dy, ok, ok, dwp, dg, ws, nbytes, z)
    assert bwd(_prob(), nbytes=16) == _lib.HMM_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(ws=z), dict(dy=z), dict(wp=ok), dict(rstd=z)):
        assert bwd(_prob(), **kw) == _lib.HMM_ERR_NULL_POINTER, kw
    assert bwd(_prob(gate_kind=2), g=ok) == _lib.HMM_ERR_NULL_POINTER
    assert bwd(_prob(), y=z, dy=z, wp=ok, dwp=ok) == _lib.HMM_ERR_BAD_SHAPE


def test_python_refuses_host_tensors_and_other_objects():
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        hmm.rms_norm(x, w)
    with pytest.raises(ValueError, match="HIP device"):
        hmm.residual_norm(x, x, w)
    with pytest.raises(TypeError, match="torch.Tensor"):
        hmm.rms_norm(x.numpy() if x.dtype != torch.bfloat16 else [1.0], w)
