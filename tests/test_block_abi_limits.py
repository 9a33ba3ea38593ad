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


def product(L, call, M=8, N=16, K=128, **kw):
    g = L.GemmArgs(M=M, N=N, K=K, lda=kw.pop("lda", K), ldb=kw.pop("ldb", K), ldd=N, A=0x1000, a_fmt=0, a_scaling=0, a_scale_inv=0x2000,
                   B=0x3000, b_fmt=0, b_scaling=0, b_scale_inv=0x4000, D=0x5000, d_dtype=0)
    e = L.EpilogueArgs(backward=0, act=0, param_dtype=0, res_scale=1.0, workspace=0x10000, workspace_bytes=1 << 62)
    for k, v in kw.items():
        setattr(e if hasattr(e, k) else g, k, v)
    return call(C.byref(g), C.byref(e))


def test_product_plan(L):
    plan = L.EpPlan()

    def ask(g, e):
        return L._L.fp8_scaled_gemm_ep_plan(g, e, C.byref(plan))

    for size, want in [((1, 4096, 4096), (L.EP_FEW_ROWS, 16, 1)), ((16, 4096, 4096), (L.EP_FEW_ROWS, 16, 1)),
                       ((8192, 8192, 8192), (L.EP_LARGE, 256, 1)), ((0, 64, 64), (L.EP_FEW_ROWS, 16, 1))]:
        assert product(L, ask, *size) == 0 and (plan.kernel, plan.tile_rows, plan.k_parts) == want
    assert product(L, ask, 8192, 8191, 8192) == 0 and plan.kernel == L.EP_TILES      # not for whole vectors
    assert product(L, ask, 64, 512, 8192) == 0 and plan.kernel == L.EP_TILES and plan.k_parts > 1
    # the workspace is not looked at; everything else is refused as by the call
    assert product(L, ask, workspace=None, workspace_bytes=0) == 0
    assert product(L, ask, K=100) == SHAPE and product(L, ask, act=9) == ARG and product(L, ask, aux=0x6001, ldaux=16) == ALIGN
    assert product(L, lambda g, e: L._L.fp8_scaled_gemm_ep_plan(g, e, None)) == NULL
    assert L._L.fp8_scaled_gemm_ep_plan(None, None, C.byref(plan)) == NULL


def test_product_grids(L):
    plan = L.EpPlan()

    def ask(g, e):
        return L._L.fp8_scaled_gemm_ep_plan(g, e, C.byref(plan))

    # a launch's threads are counted in 32 bits, its workgroups in y in 16: the join
    # of K parts takes 16 rows per workgroup
    assert product(L, ask, 1048560, 1, 8192) == 0
    for M, N, K in [(1048577, 1, 8192), (1048577, 1, 65536), (1100000, 1, 65536), (2000001, 128, 65536)]:
        assert product(L, ask, M, N, K) == 0 and plan.k_parts == 1
    n = (1 << 28) - 64
    assert product(L, ask, 16, n, 128) == 0 and product(L, ask, 16, n + 1, 128) == UNSUPPORTED
    assert product(L, ask, 17, n + 1, 128) == 0
    assert product(L, ask, 17, n + 1, 128, backward=1, dbias=0x6000) == UNSUPPORTED
    assert product(L, ask, 17, n, 128, backward=1, dbias=0x6000) == 0
    assert product(L, ask, 128, 1 << 30, 128) == 0 and product(L, ask, 129, 1 << 30, 128) == UNSUPPORTED


def test_product_inner_dimension(L):
    def call(g, e):
        return L._L.fp8_scaled_gemm_ep(g, e, None)

    assert product(L, call, K=65552) == UNSUPPORTED and product(L, call, K=65536, lda=1 << 23) == UNSUPPORTED
    plan = L.EpPlan()
    assert product(L, lambda g, e: L._L.fp8_scaled_gemm_ep_plan(g, e, C.byref(plan)), K=65536) == 0


def test_norm_gradient_without_columns(L):
    a = L.NormBwdArgs(rows=4, cols=0, kind=0, stream_dtype=0, param_dtype=1, gate=0x5000, gate_kind=2, dgate=0x6002)
    assert L._L.fp8_block_norm_bwd(C.byref(a), None) == ALIGN
    a.dgate = None
    assert L._L.fp8_block_norm_bwd(C.byref(a), None) == 0
