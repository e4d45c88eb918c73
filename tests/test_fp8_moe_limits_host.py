"""E4M3 products and encoders at the limits of one launch, whose grid may not have 2^32
threads (CPU only: what is refused is refused before a device is asked for, what is
accepted ends at the missing device)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from bit_quantized_matmul_amd import binding as B

P = ctypes.c_void_p(4096)                             # never dereferenced
NOGPU = pytest.mark.skipif(torch.cuda.is_available(), reason="would reach the device")


def gemm(m, rows):
    return B.load_library().fp8_gemm(P, P, rows, 128, P, P, m, P, 0, None)


def grouped(experts, slots, rows):
    return B.load_library().fp8_gemm_grouped(P, P, experts, rows, 128, P, P, 1, P, P, slots, P, 0, None)


def pack(rows, cols):
    return B.load_library().fp8_pack(P, 0, 1, rows, cols, P, P, None)


# tiles of 128 x 128 and, with fewer than 96 rows an expert, 64 x 128, a workgroup of 256 threads each
@pytest.mark.parametrize("call,args", [
    (gemm, (128 * 128, 1 << 24)),                     # 128 x 2^17 tiles
    (gemm, (1 << 24, 128 * 128)),
    (gemm, ((1 << 31) - 1, 1)),
    (grouped, (4096, (1 << 31) - 1, 1)),
    (grouped, (4096, 4096, 4096 * 128)),              # (64 + 4096) x 2^12 tiles
    (grouped, (1, 128 * 128, 1 << 24)),
    (pack, (1 << 24, 128 * 128)),
])
def test_more_workgroups_than_a_launch_takes(call, args):
    assert call(*args) == B.BQM_ENOTSUP


@NOGPU
@pytest.mark.parametrize("call,args", [
    (gemm, (127 * 128, 1 << 24)),
    (gemm, (1, 1 << 24)),
    (gemm, ((1 << 31) - 128, 1)),
    (grouped, (4096, 4096, 4032 * 128)),
    (grouped, (1, 126 * 128, 1 << 24)),
    (grouped, (4096, (1 << 31) - 4097 * 128, 1)),
    (pack, (1 << 24, 127 * 128)),
])
def test_as_many_as_it_takes(call, args):
    assert call(*args) == B.BQM_EDEVICE
