"""Refusals of the 8-bit float products and the mixture-of-experts calls (CPU only:
every call here is refused before it reaches a device)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from bit_quantized_matmul_amd import binding as B

P = ctypes.c_void_p(4096)                             # never dereferenced: the checks fail first
ODD = ctypes.c_void_p(4097)
OFF8 = ctypes.c_void_p(4104)                          # 8-byte aligned only
EINVAL, EALIGN, ENOTSUP = B.BQM_EINVAL, B.BQM_EALIGN, B.BQM_ENOTSUP


@pytest.fixture(scope="module")
def lib():
    return B.load_library()


@pytest.mark.parametrize("args,code", [
    ((None, 0, 1, 128, 128, 0, P, P, None), EINVAL),
    ((P, 3, 1, 128, 128, 0, P, P, None), EINVAL),
    ((P, 0, 0, 128, 128, 0, P, P, None), EINVAL),
    ((P, 0, 1, 0, 128, 0, P, P, None), EINVAL),
    ((P, 0, 2, 128, 127, 0, P, P, None), EINVAL),
    ((P, 0, 2, 128, 255, 1, P, P, None), EINVAL),
    ((P, 0, 1, (1 << 22) + 1, 1 << 23, 0, P, P, None), ENOTSUP),
    ((P, 0, 1, 128, 128, 0, OFF8, P, None), EALIGN),
    ((P, 0, 1, 128, 128, 0, P, ODD, None), EALIGN),
    ((ctypes.c_void_p(4098), 0, 1, 128, 128, 0, P, P, None), EALIGN),
    ((ODD, 1, 1, 128, 128, 0, P, P, None), EALIGN),
])
def test_quant_refuses(lib, args, code):
    assert lib.fp8_quant(*args) == code


@pytest.mark.parametrize("args,code", [
    ((P, 0, 0, 8, 128, P, P, None), EINVAL),
    ((P, 0, 1, 0, 128, P, P, None), EINVAL),
    ((P, 9, 1, 8, 128, P, P, None), EINVAL),
    ((P, 0, 4097, 8, 128, P, P, None), ENOTSUP),
    ((P, 0, 1, (1 << 24) + 1, 128, P, P, None), ENOTSUP),
    ((P, 0, 1, 1 << 24, 1 << 22, P, P, None), ENOTSUP),                  # 2^32 blocks
    ((P, 0, 1, 8, 128, OFF8, P, None), EALIGN),
])
def test_pack_refuses(lib, args, code):
    assert lib.fp8_pack(*args) == code


@pytest.mark.parametrize("args,code", [
    ((None, P, 8, 128, P, P, 1, P, 0, None), EINVAL),
    ((P, P, 8, 128, P, None, 1, P, 0, None), EINVAL),
    ((P, P, 0, 128, P, P, 1, P, 0, None), EINVAL),
    ((P, P, 8, 0, P, P, 1, P, 0, None), EINVAL),
    ((P, P, 8, 128, P, P, 0, P, 0, None), EINVAL),
    ((P, P, 8, 128, P, P, 1, P, 4, None), EINVAL),
    ((P, P, 8, (1 << 22) + 1, P, P, 1, P, 0, None), ENOTSUP),
    ((P, P, 1 << 24, 128, P, P, 1 << 16, P, 0, None), ENOTSUP),         # 2^32 tiles
    ((OFF8, P, 8, 128, P, P, 1, P, 0, None), EALIGN),
    ((P, P, 8, 128, OFF8, P, 1, P, 0, None), EALIGN),
    ((P, ODD, 8, 128, P, P, 1, P, 0, None), EALIGN),
    ((P, P, 8, 128, P, P, 1, ODD, 1, None), EALIGN),
])
def test_gemm_refuses(lib, args, code):
    assert lib.fp8_gemm(*args) == code


@pytest.mark.parametrize("args,code", [
    ((P, P, 4, 8, 128, P, P, 1, None, P, 8, P, 0, None), EINVAL),      # offsets are needed
    ((P, P, 0, 8, 128, P, P, 1, P, P, 8, P, 0, None), EINVAL),
    ((P, P, 4, 8, 128, P, P, 1, P, P, 0, P, 0, None), EINVAL),
    ((P, P, 4, 8, 128, P, P, 7, P, None, 8, P, 0, None), EINVAL),      # without row_ids slots <= m
    ((P, P, 4097, 8, 128, P, P, 1, P, P, 8, P, 0, None), ENOTSUP),
    ((P, P, 4, 8, 4096, P, P, 1 << 20, P, P, 8, P, 0, None), ENOTSUP),  # gathered rows of 2^32 bytes
    ((P, P, 4, 8, 128, P, P, 1, ODD, P, 8, P, 0, None), EALIGN),
    ((P, P, 4, 8, 128, P, P, 1, P, ODD, 8, P, 0, None), EALIGN),
])
def test_grouped_refuses(lib, args, code):
    assert lib.fp8_gemm_grouped(*args) == code


def test_route_refuses(lib):
    n = ctypes.c_int64()
    assert lib.moe_route_workspace(1, 8, 9, ctypes.byref(n)) == EINVAL
    assert lib.moe_route_workspace(1, 8, 2, None) == EINVAL
    assert lib.moe_route_workspace(1, 1025, 2, ctypes.byref(n)) == ENOTSUP
    assert lib.moe_route_workspace(1, 64, 33, ctypes.byref(n)) == ENOTSUP
    assert lib.moe_route_workspace(1 << 30, 64, 8, ctypes.byref(n)) == ENOTSUP
    assert lib.moe_route_workspace(4, 64, 8, ctypes.byref(n)) == B.BQM_OK and n.value == 0
    need = B.moe_route_workspace(4096, 64, 8)
    assert need > 0

    def call(logits=P, dtype=0, tokens=4, experts=8, stride=8, top=2, ids=P, ws=None, nws=0):
        return lib.moe_route(logits, dtype, tokens, experts, stride, top, 1, ids, P, P, P, P, ws, nws, None)

    assert call(logits=None) == EINVAL
    assert call(dtype=7) == EINVAL
    assert call(top=0) == EINVAL
    assert call(stride=7) == EINVAL
    assert call(tokens=4096, experts=64, stride=64, top=8) == EINVAL              # no workspace
    assert call(tokens=4096, experts=64, stride=64, top=8, ws=P, nws=need - 1) == EINVAL
    assert call(ids=ODD) == EALIGN
    assert call(logits=ODD, dtype=1) == EALIGN


@pytest.mark.parametrize("args,code", [
    ((None, 0, 8, 64, P, P, 4, 2, P, None), EINVAL),
    ((P, 0, 0, 64, P, P, 4, 2, P, None), EINVAL),
    ((P, 0, 8, 64, P, P, 0, 2, P, None), EINVAL),
    ((P, 3, 8, 64, P, P, 4, 2, P, None), EINVAL),
    ((P, 0, 8, (1 << 26) + 1, P, P, 4, 2, P, None), ENOTSUP),
    ((OFF8, 0, 8, 64, P, P, 4, 2, P, None), EALIGN),
    ((P, 0, 8, 64, ODD, P, 4, 2, P, None), EALIGN),
])
def test_combine_refuses(lib, args, code):
    assert lib.moe_combine(*args) == code


def test_binding_refuses_shapes_types_and_devices():
    f8, f32 = torch.float8_e4m3fn, torch.float32
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="CUDA"):
        B.fp8_quant(x)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        B.fp8_quant(x.double())
    with pytest.raises(ValueError, match="2-D"):
        B.fp8_quant(x[0])
    q, qs = torch.zeros(4, 256, dtype=f8), torch.zeros(2, 4)
    w, ws = torch.zeros(130, 256, dtype=f8), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        B.fp8_gemm(w, ws, 200, q, qs)
    with pytest.raises(ValueError, match="w must have shape"):
        B.fp8_gemm(w, ws, 300, q, qs)
    with pytest.raises(ValueError, match="w_scale"):
        B.fp8_gemm(w, ws[:1], 200, q, qs)
    with pytest.raises(ValueError, match="q_scale"):
        B.fp8_gemm(w, ws, 200, q, qs.t())
    with pytest.raises(ValueError, match="y must be"):
        B.fp8_gemm(w, ws, 200, q, qs, dtype=f32, y=torch.zeros(4, 130, dtype=torch.float16))
    with pytest.raises(ValueError, match="float32, bfloat16 or float16|CUDA"):
        B.fp8_gemm(w, ws, 200, q, qs, dtype=torch.float64)
    with pytest.raises(ValueError, match="offsets"):
        B.fp8_gemm_grouped(w[None], ws[None], 200, q, qs, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="w must have shape"):
        B.fp8_gemm_grouped(w, ws, 200, q, qs, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="row_ids"):
        B.fp8_gemm_grouped(w[None], ws[None], 200, q, qs, torch.zeros(2, dtype=torch.int32),
                           row_ids=torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="weights"):
        B.moe_combine(x, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 3))
    with pytest.raises(ValueError, match="CUDA"):
        B.moe_route(x, 2)


def test_calls_fail_loudly_without_the_extension(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "_CALLS_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(B, "_calls_module", None)
    with pytest.raises(RuntimeError, match="missing"):
        B.moe_route(torch.zeros(4, 8), 2)


def test_calls_refuse_what_is_no_tensor_or_argument():
    q, qs = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(2, 4)
    with pytest.raises(ValueError, match="w must be"):
        B.fp8_gemm(None, None, 256, q, qs)
    with pytest.raises(ValueError, match="x must be"):
        B.fp8_quant([1.0])
    with pytest.raises(ValueError, match="cols must be at least 1"):
        B.fp8_gemm(q, qs, 0, q, qs)
    with pytest.raises(TypeError):
        B.fp8_gemm(q, qs, "many", q, qs)
    with pytest.raises(ValueError, match="out of range"):
        B.fp8_gemm(q, qs, 1 << 40, q, qs)
    with pytest.raises(ValueError, match="dtype must be a torch.dtype"):
        B.fp8_gemm(torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(1, 2), 256, q, qs, dtype=7)
    with pytest.raises(ValueError, match="rows must be contiguous"):
        B.fp8_quant(torch.zeros(8, 4).t())
    with pytest.raises(ValueError, match="rows must not overlap"):
        B.fp8_quant(torch.zeros(64).as_strided((4, 16), (8, 1)))
    with pytest.raises(ValueError, match="must not be empty"):
        B.fp8_quant(torch.zeros(0, 16))
    with pytest.raises(ValueError, match="gate and up"):
        B.fp8_quant(torch.zeros(2, 15), swiglu=True)
