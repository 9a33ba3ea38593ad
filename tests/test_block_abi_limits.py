"""Sizes at the limits of the operators around the linears: every one is either
taken or refused with its documented status, on the host (these run without a
GPU; the pointers are never read)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


NULL, SHAPE, ALIGN, UNSUPPORTED, ARG = 1, 2, 3, 4, 6


@pytest.mark.parametrize("rows,cols", [(0, 32769), (1, 32769), (8, 40000), (4096, 65536), (1, 1 << 31), (1 << 40, 1 << 40)])
def test_norm_gradient_wider_than_its_rows(L, rows, cols):
    assert L._L.fp8_block_norm_bwd_workspace(rows, cols) == 0
    a = L.NormBwdArgs(rows=rows, cols=cols, kind=0, stream_dtype=0, param_dtype=1, res_scale=1, branch_scale=1, dy=0x1000,
                      lddy=cols, h=0x3000, ldh=cols, stats_h=0x4000, dx=0x7000, lddx=cols, workspace=0x9000, workspace_bytes=1 << 62)
    assert L._L.fp8_block_norm_bwd(C.byref(a), None) == UNSUPPORTED


@pytest.mark.parametrize("cols", [1, 7, 512, 513, 1024, 1025, 8192, 8193, 16385, 32768])
@pytest.mark.parametrize("rows", [0, 1, 100, 1 << 33])
def test_norm_gradient_workspace(L, rows, cols):
    n = L._L.fp8_block_norm_bwd_workspace(rows, cols)
    assert n > 0 and n % (16 * cols) == 0   # four rows of binary32 sums per workgroup
