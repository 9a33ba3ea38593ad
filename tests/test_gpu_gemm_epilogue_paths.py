"""fp8_scaled_gemm_ep on each of its kernels: values that every partial sum of a
product holds exactly, so that the outputs have to be equal and not merely near,
and products without an inner dimension."""
import pytest
import torch

from gpu_util import Guarded, say

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


@pytest.mark.parametrize("scalings", [(0, 0), (5, 5), (1, 2), (1, 1), (2, 2), (3, 4), (0, 2), (1, 0), (0, 3), (0, 4), (3, 0), (4, 0)])
@pytest.mark.parametrize("rows", [5, 40, 300])
def test_no_inner_dimension_and_no_scales(L, rows, scalings):
    """K = 0: a sum of nothing, for which scales need not be there."""
    say("no K", rows, scalings)
    N, g = 136, torch.Generator(device="cuda").manual_seed(rows)
    A, B = torch.empty((rows, 0), dtype=U8, device="cuda"), torch.empty((N, 0), dtype=U8, device="cuda")
    bias, res = torch.randn(N, generator=g, device="cuda"), torch.randn((rows, N), generator=g, device="cuda")
    D, aux = Guarded((rows, N), F32), Guarded((rows, N), BF)
    L.fp8_scaled_gemm_ep(A, 0, scalings[0], None, B, 0, scalings[1], None, D.t, bias=bias, act=L.ACT_RELU, aux=aux.t, residual=res)
    torch.cuda.synchronize()
    D.check(), aux.check()
    assert torch.equal(D.t, bias.clamp(min=0) + res)
    assert torch.equal(aux.t, bias.to(BF).expand(rows, N))
    db = torch.full((N,), 7.0, device="cuda")
    L.fp8_scaled_gemm_ep(A, 1, scalings[0], None, B, 0, scalings[1], None, D.t, act=L.ACT_SILU, aux=aux.t, backward=True, dbias=db)
    torch.cuda.synchronize()
    D.check()
    assert bool((D.t == 0).all()) and bool((db == 0).all())


# ---- every kernel, with values that are sums of few small integers: products and
# column sums are exact in binary32 whatever their order (all partial sums are
# integers below 2^24: K 2 2 4 4 at most for a product, and what is added up in a
# column is some 2^11 times less), so one lost row, part of K or bit shows

FEW, TILES, LARGE = 0, 1, 2
# rows, columns, K, scalings, kernel, rows of its tiles, whether K is cut
PATHS = [
    (3, 1000, 4112, (0, 0), FEW, 16, False), (16, 520, 2064, (5, 5), FEW, 16, False), (1, 264, 48, (0, 5), FEW, 16, False),
    (13, 264, 4096, (1, 2), FEW, 16, False), (7, 328, 2048, (1, 1), FEW, 16, False), (16, 136, 1024, (3, 4), FEW, 16, False),
    (33, 520, 656, (0, 0), TILES, 32, False), (64, 512, 8192, (5, 0), TILES, 32, True), (300, 520, 4112, (5, 5), TILES, 32, True),
    (130, 264, 2048, (1, 2), TILES, 32, True), (130, 264, 2048, (3, 4), TILES, 32, True), (130, 264, 2048, (1, 1), TILES, 32, True),
    (33, 520, 640, (0, 4), TILES, 32, False),
    (1037, 1999, 2320, (5, 5), TILES, 64, False), (1037, 1999, 2304, (1, 2), TILES, 64, False), (1500, 2000, 384, (3, 4), TILES, 64, False),
    (1500, 2000, 384, (2, 1), TILES, 64, False), (300, 1000, 4096, (1, 2), TILES, 64, True), (300, 1000, 4096, (3, 3), TILES, 64, True),
    (2050, 4103, 656, (0, 0), TILES, 128, False), (1100, 4104, 512, (5, 5), TILES, 128, False), (2048, 4096, 512, (1, 2), TILES, 128, False),
    (2048, 4096, 512, (1, 1), TILES, 128, False), (2048, 4096, 512, (2, 2), TILES, 128, False), (2048, 4096, 512, (3, 4), TILES, 128, False),
    (2048, 4096, 512, (4, 3), TILES, 128, False), (2048, 4096, 512, (0, 2), TILES, 128, False),
    (2050, 4104, 640, (0, 0), LARGE, 256, False), (2050, 4104, 656, (0, 0), LARGE, 256, False), (2050, 4104, 640, (5, 5), LARGE, 256, False),
    (2050, 4104, 656, (5, 5), LARGE, 256, False), (2050, 4104, 656, (0, 5), LARGE, 256, False), (2050, 4104, 640, (1, 2), LARGE, 256, False),
    (2050, 4104, 640, (3, 4), LARGE, 256, False)]
CODE = {0: {0: 0x00, 1: 0x38, 2: 0x40, -1: 0xB8, -2: 0xC0}, 1: {0: 0x00, 1: 0x3C, 2: 0x40, -1: 0xBC, -2: 0xC0}}


def small(g, rows, K, fmt, scaling):
    """Codes and inverse scales (1, 2 or 4) of a [rows][K] operand, and its values in 64 bits."""
    v = torch.tensor([0, 0, 0, 0, 1, -1, 2, -2], device="cuda")[torch.randint(0, 8, (rows, K), generator=g, device="cuda")]
    table = torch.zeros(5, dtype=U8, device="cuda")
    for value, code in CODE[fmt].items():
        table[value + 2] = code
    nkb = -(-K // 128)
    shape = {0: (1,), 5: (rows,), 1: (nkb, rows), 3: (nkb, rows)}.get(scaling, (nkb, -(-rows // 128)))
    s = torch.randint(0, 3, shape, generator=g, device="cuda").float().exp2()
    wide = v.double()
    if scaling in (0, 5):
        wide = wide * (s if scaling == 0 else s[:, None]).double()
    else:
        seg = s.double().t().repeat_interleave(128, 1)
        wide = wide * (seg if scaling in (1, 3) else seg.repeat_interleave(128, 0)[:rows])
    return table[v + 2], s, wide


@pytest.fixture
def taken(L, monkeypatch):
    """The kernels that the calls of a test have taken."""
    import ctypes as C
    call, seen = L._L.fp8_scaled_gemm_ep, []

    def spy(gemm, ep, stream):
        plan = L.EpPlan()
        assert L._L.fp8_scaled_gemm_ep_plan(gemm, ep, C.byref(plan)) == 0
        seen.append((plan.kernel, plan.tile_rows, plan.k_parts > 1))
        return call(gemm, ep, stream)

    monkeypatch.setattr(L._L, "fp8_scaled_gemm_ep", spy)
    return seen


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("out", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("backward", [False, True])
def test_exact_on_each_kernel(L, taken, path, out, backward):
    M, N, K, (asc, bsc), *kernel = path
    say("exact", path, out, backward)
    g = torch.Generator(device="cuda").manual_seed(M + N + K + asc)
    A, sa, a = small(g, M, K, int(backward), asc)
    B, sb, b = small(g, N, K, 0, bsc)
    v = torch.matmul(a, b.t())
    D = Guarded((M, N), {"f32": F32, "bf16": BF, "fp8": U8}[out])
    amax, kw = Guarded((1,), F32), {"act": L.ACT_RELU, "backward": backward}
    fmt, f8, top, scale = (1, torch.float8_e5m2, 57344.0, 4.0) if backward else (0, torch.float8_e4m3fn, 448.0, 0.25)
    if out == "fp8":
        D_t = Guarded((N, M), U8)
        kw.update(d_fmt=fmt, d_scale=torch.full((1,), scale, device="cuda"), D_t=D_t.t)
    if backward:
        kw["aux"] = torch.randn((M, N), generator=g, device="cuda").to(BF)
        db = Guarded((N,), F32)
        kw["dbias"] = db.t
        want = v * (kw["aux"] > 0)
    else:
        bias = torch.randint(-8, 9, (N,), generator=g, device="cuda").float()
        res = torch.randint(-64, 65, (M, N), generator=g, device="cuda").to(F32 if out == "f32" else BF)
        aux = Guarded((M, N), BF)
        kw.update(bias=bias, residual=res, res_scale=0.5, aux=aux.t)
        u = v + bias.double()
        want = u.clamp(min=0) + 0.5 * res.double()
    L.fp8_scaled_gemm_ep(A, int(backward), asc, sa, B, 0, bsc, sb, D.t, d_amax=amax.t, **kw)
    torch.cuda.synchronize()
    assert taken == [tuple(kernel)]
    D.check(), amax.check()
    if out == "fp8":
        D_t.check()
        assert torch.equal(D.t.view(f8).float(), (want * scale).clamp(-top, top).float().to(f8).float())
        assert torch.equal(D_t.t, D.t.t())
    else:
        assert torch.equal(D.t, want.float().to(D.t.dtype))
    assert float(amax.t) == float((want.float().to(BF) if out == "bf16" else want.float()).abs().max())
    if backward:
        db.check()
        assert torch.equal(db.t, want.sum(0).float())
    else:
        aux.check()
        assert torch.equal(aux.t, u.float().to(BF))


@pytest.mark.parametrize("path", PATHS)
def test_bias_gradient_is_the_sum_of_its_own_outputs(L, taken, path):
    """Random values, a smooth activation: D holds, unrounded, what the bias
    gradient adds up, at most 64 values one after the other on the way."""
    M, N, K, (asc, bsc), *kernel = path
    say("column sums", path)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    A, sa, _ = small(g, M, K, 1, asc)
    B, sb, _ = small(g, N, K, 0, bsc)
    D, db = Guarded((M, N), F32), Guarded((N,), F32)
    L.fp8_scaled_gemm_ep(A, 1, asc, sa, B, 0, bsc, sb, D.t, act=L.ACT_GELU_TANH, backward=True, dbias=db.t,
                         aux=torch.randn((M, N), generator=g, device="cuda").to(BF))
    torch.cuda.synchronize()
    assert taken == [tuple(kernel)]
    D.check(), db.check()
    d = D.t.double()
    assert bool(((db.t.double() - d.sum(0)).abs() <= 64 * 2.0 ** -24 * d.abs().sum(0)).all())
