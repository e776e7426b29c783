"""Refusals of moe_decode and of the FP8 block product, all on the host (no GPU is touched)."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_int32_amd as hmm
from mixture_experts_ffn_int32_amd import _lib

Z, OK, BAD = ctypes.c_void_p(0), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _prob(**kw):
    d = dict(T=4, H=128, I=128, E=8, K=2, weight_dtype=_lib.HMM_BF16, router_dtype=_lib.HMM_BF16, flags=0)
    d.update(kw)
    return _lib.DecodeProblem(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), _lib.HMM_ERR_BAD_SHAPE), (dict(T=65), _lib.HMM_ERR_UNSUPPORTED), (dict(E=0), _lib.HMM_ERR_BAD_SHAPE),
    (dict(E=1025), _lib.HMM_ERR_BAD_SHAPE), (dict(K=0), _lib.HMM_ERR_BAD_SHAPE), (dict(K=17), _lib.HMM_ERR_BAD_SHAPE),
    (dict(H=96), _lib.HMM_ERR_BAD_SHAPE), (dict(I=0), _lib.HMM_ERR_BAD_SHAPE), (dict(H=65600), _lib.HMM_ERR_BAD_SHAPE),
    (dict(weight_dtype=_lib.HMM_FP8_E4M3), _lib.HMM_ERR_BAD_DTYPE), (dict(router_dtype=_lib.HMM_FP8_E4M3), _lib.HMM_ERR_BAD_DTYPE),
    (dict(weight_dtype=_lib.HMM_FP8_E4M3_BLOCK, H=192), _lib.HMM_ERR_BAD_SHAPE),
    (dict(weight_dtype=_lib.HMM_FP8_E4M3_BLOCK, I=64), _lib.HMM_ERR_BAD_SHAPE), (dict(flags=2), _lib.HMM_ERR_BAD_SHAPE),
    (dict(), _lib.HMM_OK), (dict(T=0), _lib.HMM_OK), (dict(T=64, weight_dtype=_lib.HMM_FP8_E4M3_BLOCK), _lib.HMM_OK)])
def test_decode_problem(lib, kw, status):
    n = ctypes.c_size_t()
    assert lib.hmm_moe_decode_sizes(ctypes.byref(_prob(**kw)), ctypes.byref(n)) == status


def test_decode_pointers(lib):
    def call(p, nbytes=1 << 40, **kw):
        a = dict(x=OK, router=Z, ids=OK, w=OK, up=OK, ud=Z, down=OK, dd=Z, y=OK, ws=OK)
        a.update(kw)
        return lib.hmm_moe_decode(ctypes.byref(p), a["x"], a["router"], a["ids"], a["w"], a["up"], a["ud"], a["down"], a["dd"],
                                  a["y"], a["ws"], nbytes, Z)
    for k in ("x", "ids", "w", "up", "down", "y", "ws"):
        assert call(_prob(), **{k: Z}) == _lib.HMM_ERR_NULL_POINTER, k
        assert call(_prob(), **{k: BAD}) == _lib.HMM_ERR_MISALIGNED, k
    assert call(_prob(), router=BAD) == _lib.HMM_ERR_MISALIGNED
    fp8 = dict(weight_dtype=_lib.HMM_FP8_E4M3_BLOCK)
    assert call(_prob(**fp8), dd=OK) == _lib.HMM_ERR_NULL_POINTER
    assert call(_prob(**fp8), ud=OK) == _lib.HMM_ERR_NULL_POINTER
    assert call(_prob(), nbytes=8) == _lib.HMM_ERR_WORKSPACE_TOO_SMALL
    assert call(_prob(E=2, K=3), router=OK) == _lib.HMM_ERR_BAD_SHAPE
    assert call(_prob(T=0), x=Z, ids=Z, w=Z, y=Z, ws=Z) == _lib.HMM_OK


@pytest.mark.parametrize("T,H,N,status", [
    (-1, 128, 128, _lib.HMM_ERR_BAD_SHAPE), (1 << 31, 128, 128, _lib.HMM_ERR_BAD_SHAPE), (4, 64, 128, _lib.HMM_ERR_BAD_SHAPE),
    (4, 192, 128, _lib.HMM_ERR_BAD_SHAPE), (4, 65664, 128, _lib.HMM_ERR_BAD_SHAPE), (4, 128, 8, _lib.HMM_ERR_BAD_SHAPE),
    (4, 128, 0, _lib.HMM_ERR_BAD_SHAPE), (4, 128, 262160, _lib.HMM_ERR_BAD_SHAPE), (1 << 30, 128, 128, _lib.HMM_ERR_UNSUPPORTED),
    (4, 128, 16, _lib.HMM_OK), (0, 128, 16, _lib.HMM_OK)])
def test_block_dims(lib, T, H, N, status):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.hmm_linear_fp8_block_sizes(T, H, N, ctypes.byref(a), ctypes.byref(b)) == status
    assert lib.hmm_matmul_fp8_block(Z, Z, OK, OK, T, H, N, Z, Z) == (status or (_lib.HMM_ERR_NULL_POINTER if T else 0))  # no data pointers: a valid shape is refused for them


def test_block_pointers(lib):
    T, H, N = 100, 256, 256
    assert lib.hmm_quant_block(OK, 1, H, N, Z, Z, OK, Z) == _lib.HMM_ERR_NULL_POINTER
    assert lib.hmm_quant_block(OK, 1, H, N, OK, BAD, OK, Z) == _lib.HMM_ERR_MISALIGNED
    assert lib.hmm_quant_block(OK, 0, H, N, OK, Z, OK, Z) == _lib.HMM_ERR_BAD_SHAPE
    assert lib.hmm_linear_fp8_block(OK, OK, OK, T, H, N, OK, Z, 0, Z) == _lib.HMM_ERR_NULL_POINTER
    assert lib.hmm_linear_fp8_block(OK, OK, OK, T, H, N, OK, OK, 16, Z) == _lib.HMM_ERR_WORKSPACE_TOO_SMALL
    assert lib.hmm_linear_fp8_block(BAD, OK, OK, 4, H, N, OK, Z, 0, Z) == _lib.HMM_ERR_MISALIGNED

    def grad(T=T, N=N, dy=OK, x=OK, q=OK, ds=OK, dx=OK, dw=OK, ws=OK, nbytes=1 << 40):
        return lib.hmm_linear_fp8_block_grad(dy, x, q, ds, T, H, N, dx, dw, ws, nbytes, Z)
    assert grad(N=144) == _lib.HMM_ERR_BAD_SHAPE
    for kw in (dict(dy=Z), dict(x=Z), dict(q=Z), dict(ds=Z), dict(ws=Z)):
        assert grad(**kw) == _lib.HMM_ERR_NULL_POINTER, kw
    assert grad(nbytes=8) == _lib.HMM_ERR_WORKSPACE_TOO_SMALL
    assert grad(T=1 << 24) == _lib.HMM_ERR_UNSUPPORTED  # operands of 4 GiB and more


def test_python_refuses_host_tensors_and_other_objects():
    x, w = torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((128, 128), dtype=torch.bfloat16)
    for f in (lambda: hmm.quantize_block(w), lambda: hmm.linear_fp8_block(x, w), lambda: hmm.matmul_fp8_block(x.view(torch.uint8), x, w, w),
              lambda: hmm.moe_decode(x, w[None], w[None], top_k=1, router_weight=w)):
        with pytest.raises(ValueError, match="HIP device"):
            f()
    with pytest.raises(TypeError, match="torch.Tensor"):
        hmm.moe_decode(None, w, w)
