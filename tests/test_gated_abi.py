"""Refusals of the gated feed-forward pair and of 8-bit checkpoints: every bad
call returns its status on the host, before any launch (these run without a GPU;
the pointers are never read)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


NULL, SHAPE, ALIGN, UNSUPPORTED, ARG = 1, 2, 3, 4, 6


def gated(L, ep=None, call=None, **kw):
    g = L.GemmArgs(M=8, N=48, K=128, lda=128, ldb=128, ldd=96, A=0x1000, a_fmt=0, a_scaling=0, a_scale_inv=0x2000, B=0x3000,
                   b_fmt=0, b_scaling=0, b_scale_inv=0x4000, D=0x5000, d_dtype=0)
    for k, v in kw.items():
        setattr(g, k, v)
    e = L.GatedArgs(backward=0, act=4, param_dtype=0, workspace=0x10000, workspace_bytes=1 << 62)
    for k, v in (ep or {}).items():
        setattr(e, k, v)
    return (call or (lambda a, b: L._L.fp8_gated_linear(a, b, None)))(C.byref(g), C.byref(e))


AUX = dict(aux=0x6000, ldaux=96)
CK = dict(ck=0x6001, ldck=96, ck_exp=0x7001, ldexp=4)
BACK = dict(backward=1, **AUX)


@pytest.mark.parametrize("kw,ep,status", [
    (dict(M=-1), {}, SHAPE), (dict(N=-1), {}, SHAPE), (dict(K=100), {}, SHAPE), (dict(a_fmt=2), {}, ARG), (dict(A=None), {}, NULL),
    (dict(D=None), {}, NULL), (dict(accumulate=1, d_dtype=1), {}, UNSUPPORTED), (dict(a_scaling=5, b_scaling=2), {}, UNSUPPORTED),
    (dict(lda=1 << 24), {}, UNSUPPORTED), (dict(ldb=1 << 24), {}, UNSUPPORTED), (dict(K=65552, lda=65552, ldb=65552), {}, UNSUPPORTED),
    (dict(a_fmt=1), {}, UNSUPPORTED), (dict(b_fmt=1), {}, UNSUPPORTED), (dict(b_fmt=1), BACK, UNSUPPORTED),
    (dict(N=(1 << 26) + 1, ldd=1 << 28), {}, UNSUPPORTED), (dict(M=1 << 28, N=1 << 16), {}, SHAPE), (dict(M=1 << 28, N=1 << 16, ldd=1 << 17), {}, UNSUPPORTED),
    (dict(D_t=0x6000), {}, ARG), (dict(d_dtype=2), {}, NULL), (dict(d_dtype=2, d_scale=0x7000, D_t=0x6000, ldt=7), {}, SHAPE),
    ({}, dict(act=5), ARG), ({}, dict(act=-1), ARG), ({}, dict(backward=2), ARG), ({}, dict(param_dtype=2), ARG), ({}, dict(dbias=0x6000), ARG),
    ({}, dict(BACK, bias=0x6000), ARG), ({}, dict(BACK, **CK), ARG), ({}, dict(backward=1), NULL),
    ({}, dict(CK, ck_exp=None), NULL), ({}, dict(CK, ck=None), NULL), ({}, dict(AUX, ldaux=95), SHAPE), ({}, dict(CK, ldck=95), SHAPE),
    ({}, dict(CK, ldexp=3), SHAPE), (dict(ldd=95), BACK, SHAPE), (dict(ldd=47), {}, SHAPE), ({}, dict(AUX, aux=0x6001), ALIGN),
    ({}, dict(bias=0x6001), ALIGN), ({}, dict(BACK, dbias=0x6001), ALIGN), ({}, dict(bias=0x6002, param_dtype=1), ALIGN),
    (dict(M=64, N=512, K=8192, lda=8192, ldb=8192, ldd=512), dict(workspace=None), NULL), ({}, dict(BACK, workspace_bytes=8), SHAPE),
    ({}, dict(workspace=0x10008), ALIGN)])
def test_gated(L, kw, ep, status):
    assert gated(L, ep, **kw) == status


def test_nothing_to_do(L):
    assert gated(L, N=0, A=None, B=None, D=None) == 0
    assert gated(L, M=0, A=None, B=None, D=None) == 0
    assert L._L.fp8_gated_linear(None, None, None) == NULL
    assert L._L.fp8_gated_linear_plan(None, None, None) == NULL


def test_plan_and_workspace(L):
    plan = L.EpPlan()

    def ask(g, e):
        return L._L.fp8_gated_linear_plan(g, e, C.byref(plan))

    wide = dict(K=4096, lda=4096, ldb=4096, N=4096, ldd=8192)
    assert gated(L, None, ask, M=1, **wide) == 0 and plan.kernel == L.EP_FEW_ROWS
    assert gated(L, None, ask, M=16, **wide) == 0 and plan.kernel == L.EP_FEW_ROWS
    # the few-row kernel has no whole blocks of a checkpoint to write; it reads one as well as BF16
    kept = dict(ck=0x6000, ldck=8192, ck_exp=0x7000, ldexp=256)
    assert gated(L, kept, ask, M=1, **wide) == 0 and plan.kernel == L.EP_TILES
    assert gated(L, dict(kept, backward=1), ask, M=1, **wide) == 0 and plan.kernel == L.EP_FEW_ROWS
    assert gated(L, None, lambda g, e: L._L.fp8_gated_linear_plan(g, e, None)) == NULL
    assert gated(L, dict(act=9), ask) == ARG
    # one size for every form of a call
    for M, F, K in [(1, 4096, 4096), (16, 512, 8192), (64, 512, 8192), (300, 1000, 4096), (8192, 28672, 8192)]:
        for a, b in [(0, 0), (5, 5), (1, 2), (3, 4)]:
            for back in (0, 1):
                need = L._L.fp8_gated_linear_workspace(M, F, K, a, b, back)
                for form in ({}, CK, AUX):
                    ep = dict(form, backward=back)
                    ep.update({k: v for k, v in (("ldck", 2 * F), ("ldaux", 2 * F), ("ldexp", 2 * -(-F // 32)))})
                    if back and not form:
                        continue
                    kw = dict(M=M, N=F, K=K, lda=K, ldb=K, ldd=2 * F, a_scaling=a, b_scaling=b)
                    assert gated(L, ep, ask, **kw) == 0
                    if plan.kernel != L.EP_FEW_ROWS and plan.k_parts > 1:
                        assert need >= plan.k_parts * M * (F if back else 2 * F) * 4
                    if back:
                        assert need >= -(-M // (2 * plan.tile_rows)) * 2 * F * 4
                    assert need == 0 or gated(L, dict(ep, workspace_bytes=need - 1), **kw) == SHAPE
    for bad in [(-1, 8, 16), (8, -1, 16), (8, 8, -1), (8, (1 << 26) + 1, 16)]:
        assert L._L.fp8_gated_linear_workspace(*bad, 0, 0, 0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(cols=-1), SHAPE), (dict(dtype=2), ARG), (dict(x=None), NULL), (dict(ck=None), NULL), (dict(exp=None), NULL),
    (dict(ldx=69), SHAPE), (dict(ldck=69), SHAPE), (dict(ldexp=2), SHAPE), (dict(x=0x1001), ALIGN), (dict(x=0x1002, dtype=1), ALIGN),
    (dict(cols=(1 << 28) + 1, ldx=1 << 30, ldck=1 << 30, ldexp=1 << 30), UNSUPPORTED), (dict(rows=0, x=None), 0),
    (dict(cols=0, ck=None), 0)])
def test_checkpoint(L, kw, status):
    a = dict(dict(x=0x1000, dtype=0, rows=4, cols=70, ldx=70, ck=0x2001, ldck=70, exp=0x3001, ldexp=3), **kw)
    x, dt, r, c, ldx, ck, ldck, exp, lde = a.values()
    assert L._L.fp8_checkpoint_save(x, dt, r, c, ldx, ck, ldck, exp, lde, None) == status
    assert L._L.fp8_checkpoint_load(ck, ldck, exp, lde, r, c, x, dt, ldx, None) == status


def test_binding_refuses(L):
    u8, bf = torch.uint8, torch.bfloat16
    A, B, D = torch.zeros((4, 128), dtype=u8), torch.zeros((64, 128), dtype=u8), torch.zeros((4, 32), dtype=bf)
    with pytest.raises(TypeError):
        L.fp8_gated_linear(A, 0, 0, None, B, 0, 0, None, D)                       # host tensors
    with pytest.raises(ValueError):
        L.fp8_gated_linear(A, 0, 0, None, B[:63], 0, 0, None, D)                  # half a pair
    with pytest.raises(TypeError):
        L.fp8_gated_linear(A, 0, 0, None, B, 0, 0, None, D.half())
    with pytest.raises(ValueError):
        L.fp8_gated_linear(A, 0, 0, None, B, 0, 0, None, D.to(u8))                # codes of which format?
    with pytest.raises(TypeError):
        L.fp8_checkpoint_save(torch.zeros((2, 64)), torch.zeros((2, 64), dtype=u8), torch.zeros((2, 2), dtype=u8))
    with pytest.raises(ValueError):
        L.fp8_checkpoint_save(torch.zeros(64), None, None)
    with pytest.raises(ValueError):
        L.fp8_checkpoint_load(None, None, torch.zeros((2, 64)))
    with pytest.raises(TypeError):
        L.fp8_checkpoint_load(torch.zeros((2, 64), dtype=u8), torch.zeros((2, 2)), torch.zeros((2, 64)))
