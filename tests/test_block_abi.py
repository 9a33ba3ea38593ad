"""Refusals of the operators around the linears: every bad call returns its
status on the host, before any launch (these run without a GPU; the pointers
are never read)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


NULL, SHAPE, ALIGN, UNSUPPORTED, ARG = 1, 2, 3, 4, 6


def norm(L, **kw):
    a = L.NormArgs(rows=4, cols=64, kind=0, stream_dtype=0, param_dtype=1, eps=1e-6, res_scale=1, branch_scale=1,
                   x=0x1000, ldx=64, z=0x2000, ldz=64, h=0x3000, ldh=64, y=0x4000, ldy=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return L._L.fp8_block_norm(C.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(kind=2), ARG), (dict(stream_dtype=2), ARG), (dict(param_dtype=-1), ARG),
    (dict(gate_kind=4), ARG), (dict(gate_act=3), ARG), (dict(gate=0x5000), ARG), (dict(gate_kind=1), ARG),
    (dict(gate=0x5000, gate_kind=1, z=None, h=None), ARG), (dict(b_post=0x5000), ARG), (dict(b_pre=0x5000), ARG),
    (dict(cols=40000, ldx=40000, ldz=40000, ldh=40000, ldy=40000), UNSUPPORTED), (dict(x=None), NULL), (dict(h=None), NULL),
    (dict(z=None), ARG), (dict(z=None, h=None, y=None), ARG), (dict(ldx=63), SHAPE), (dict(ldz=63), SHAPE), (dict(ldh=63), SHAPE),
    (dict(ldy=63), SHAPE), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(x=0x1001), ALIGN), (dict(z=0x2001), ALIGN),
    (dict(w_pre=0x5002), ALIGN), (dict(stats_z=0x5002), ALIGN), (dict(gate=0x5000, gate_kind=3, ldg=60), SHAPE),
    (dict(gate=0x5002, gate_kind=2), ALIGN), (dict(stream_dtype=1, x=0x1002), ALIGN),
    (dict(y8=0x6000, ldy8=64), NULL), (dict(y8=0x6000, ldy8=63, y8_scale=0x7000), SHAPE), (dict(y8=0x6000, ldy8=64, y8_format=2), ARG),
    (dict(y8=0x6000, ldy8=64, y8_scaling=2), UNSUPPORTED), (dict(y8=0x6000, ldy8=64, y8_scaling=3), UNSUPPORTED),
    (dict(y8=0x6000, ldy8=64, y8_scaling=5), NULL), (dict(y8=0x6000, ldy8=64, y8_scaling=1), NULL),
    (dict(y8=0x6000, ldy8=64, y8_scale=0x7002), ALIGN), (dict(rows=0), 0), (dict(cols=0), 0)])
def test_norm(L, kw, status):
    assert norm(L, **kw) == status


def norm_bwd(L, **kw):
    need = L._L.fp8_block_norm_bwd_workspace(4, 64)
    a = L.NormBwdArgs(rows=4, cols=64, kind=0, stream_dtype=0, param_dtype=1, res_scale=1, branch_scale=1, dy=0x1000, lddy=64,
                      dh=0x2000, lddh=64, h=0x3000, ldh=64, stats_h=0x4000, z=0x5000, ldz=64, stats_z=0x6000, dx=0x7000,
                      lddx=64, dz=0x8000, lddz=64, workspace=0x9000, workspace_bytes=need)
    for k, v in kw.items():
        setattr(a, k, v)
    return L._L.fp8_block_norm_bwd(C.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(kind=5), ARG), (dict(h=None), NULL), (dict(stats_h=None), NULL), (dict(stats_z=None), NULL),
    (dict(dy=None, dw_pre=0xA000), ARG), (dict(z=None, stats_z=None), ARG), (dict(dgate=0xA000), ARG),
    (dict(dy=None, dh=None), NULL), (dict(lddy=1), SHAPE), (dict(lddh=1), SHAPE), (dict(lddx=1), SHAPE), (dict(lddz=1), SHAPE),
    (dict(db_pre=0xA000), ARG), (dict(db_post=0xA000), ARG), (dict(workspace=None), NULL), (dict(workspace_bytes=16), SHAPE),
    (dict(workspace=0x9008), ALIGN), (dict(dw_pre=0xA002), ALIGN), (dict(dx=0x7001), ALIGN), (dict(cols=0), 0)])
def test_norm_bwd(L, kw, status):
    assert norm_bwd(L, **kw) == status


def gemm_ep(L, ep=None, **kw):
    g = L.GemmArgs(M=8, N=16, K=128, lda=128, ldb=128, ldd=16, A=0x1000, a_fmt=0, a_scaling=0, a_scale_inv=0x2000, B=0x3000,
                   b_fmt=0, b_scaling=0, b_scale_inv=0x4000, D=0x5000, d_dtype=0)
    for k, v in kw.items():
        setattr(g, k, v)
    e = L.EpilogueArgs(backward=0, act=0, param_dtype=0, res_scale=1.0, workspace=0x10000, workspace_bytes=1 << 40)
    for k, v in (ep or {}).items():
        setattr(e, k, v)
    return L._L.fp8_scaled_gemm_ep(C.byref(g), C.byref(e), None)


@pytest.mark.parametrize("kw,ep,status", [
    (dict(M=-1), {}, SHAPE), (dict(K=100), {}, SHAPE), (dict(a_fmt=2), {}, ARG), (dict(A=None), {}, NULL),
    (dict(accumulate=1, d_dtype=1), {}, UNSUPPORTED), (dict(a_scaling=5, b_scaling=2), {}, UNSUPPORTED),
    (dict(lda=1 << 24), {}, UNSUPPORTED), (dict(D_t=0x6000), {}, ARG), (dict(d_dtype=2), {}, NULL), ({}, dict(act=5), ARG),
    ({}, dict(backward=2), ARG), ({}, dict(param_dtype=3), ARG), ({}, dict(residual_dtype=3), ARG),
    ({}, dict(backward=1, bias=0x6000), ARG), ({}, dict(backward=1, residual=0x6000, ldres=16), ARG), ({}, dict(dbias=0x6000), ARG),
    ({}, dict(backward=1, act=1), NULL), ({}, dict(aux=0x6000, ldaux=15), SHAPE),
    (dict(d_dtype=2, d_scale=0x7000), dict(residual=0x6000, ldres=16, residual_dtype=1), UNSUPPORTED), ({}, dict(residual=0x6000, ldres=15), SHAPE),
    ({}, dict(workspace=None), NULL), ({}, dict(workspace_bytes=8), SHAPE), ({}, dict(workspace=0x10008), ALIGN),
    ({}, dict(bias=0x6001), ALIGN), ({}, dict(aux=0x6001, ldaux=16), ALIGN), (dict(M=0), {}, 0)])
def test_gemm_ep(L, kw, ep, status):
    if status == 0 and not torch.cuda.is_available():
        kw = dict(kw, N=0)
    assert gemm_ep(L, ep, **kw) == status


def test_gemm_ep_null(L):
    assert L._L.fp8_scaled_gemm_ep(None, None, None) == NULL
    assert L._L.fp8_block_norm(None, None) == NULL
    assert L._L.fp8_block_norm_bwd(None, None) == NULL
    assert L._L.fp8_rope(None, None) == NULL


def rope(L, **kw):
    a = L.RopeArgs(tokens=4, q_heads=2, k_heads=1, dim=64, pairs=32, dtype=0, layout=0, inverse=0, scale=1.0, freqs=0x1000,
                   positions=0x2000, positions_i64=1, q=0x3000, q_token_stride=128, q_head_stride=64, k=0x4000,
                   k_token_stride=64, k_head_stride=64, q_out=0x5000, q_out_token_stride=128, q_out_head_stride=64, k_out=0x6000,
                   k_out_token_stride=64, k_out_head_stride=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return L._L.fp8_rope(C.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), SHAPE), (dict(pairs=33), SHAPE), (dict(dtype=2), ARG), (dict(layout=2), ARG), (dict(inverse=2), ARG),
    (dict(positions_i64=2), ARG), (dict(q=None), NULL), (dict(q_out=None), NULL), (dict(k_out=None), NULL), (dict(freqs=None), NULL),
    (dict(freqs=0x1004), ALIGN), (dict(positions=0x2004), ALIGN), (dict(q=0x3001), ALIGN), (dict(dim=4096, pairs=1025), UNSUPPORTED),
    (dict(q_heads=65535), UNSUPPORTED), (dict(tokens=1 << 24), UNSUPPORTED), (dict(tokens=0), 0), (dict(dim=0, pairs=0), 0)])
def test_rope(L, kw, status):
    assert rope(L, **kw) == status


@pytest.mark.parametrize("a,status", [
    ((0x1000, -1, 1e4, 0, 1, 1, 1, 2), SHAPE), ((0x1000, 4, 1e4, 4, 1, 1, 1, 2), ARG), ((0x1000, 4, 0.0, 0, 1, 1, 1, 2), ARG),
    ((0x1000, 4, 1e4, 1, 0.0, 1, 1, 2), ARG), ((0x1000, 4, 1e4, 3, 2, 0, 1, 2), ARG), ((0x1000, 4, 1e4, 3, 2, 8192, 2, 2), ARG),
    ((None, 4, 1e4, 0, 1, 1, 1, 2), NULL), ((0x1004, 4, 1e4, 0, 1, 1, 1, 2), ALIGN), ((None, 0, 1e4, 0, 1, 1, 1, 2), 0)])
def test_rope_freqs(L, a, status):
    assert L._L.fp8_rope_freqs(*a, None) == status


def test_binding_refuses_host_tensors(L):
    x = torch.zeros((4, 64))
    with pytest.raises(TypeError):
        L.fp8_block_norm(x, y=x.to(torch.bfloat16))
    with pytest.raises(ValueError):
        L.fp8_block_norm(torch.zeros(4))
    with pytest.raises(TypeError):
        L.fp8_rope(torch.zeros((2, 2, 8)), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(TypeError):
        L.fp8_scaled_gemm_ep(torch.zeros((2, 16), dtype=torch.uint8), 0, 0, None, torch.zeros((2, 16), dtype=torch.uint8), 0, 0, None,
                             torch.zeros((2, 2)))
