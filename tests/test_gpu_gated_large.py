"""fp8_gated_linear on its large tiles (256 x 256 and 160 x 256): values that are sums of
few small integers come out exactly, at the tiles' edges, on strided rows that start on a
dword, and beside memory that stays as it was; which kernel is taken is checked."""
import pytest
import torch

import gated_ref as G
import test_gpu_gated as T
from gpu_util import Guarded, say
from test_gpu_gated import L, taken      # noqa: F401  (fixtures)
from test_gpu_gemm_epilogue_paths import small

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8

# rows, outputs, K, scalings, direction, rows of the tiles.  FP8 output takes the large
# kernels where D_t's rows start on a dword: an even number of rows, four to a dword.
# (3552 outputs: a last tile of 192 columns forward; 4128: of 32 backward; 2052 rows: four in it.)
PATHS = [
    (2052, 3584, 640, (0, 0), False, 256), (2052, 3552, 656, (0, 0), False, 256), (2176, 3552, 640, (5, 5), False, 256),
    (2180, 3552, 1296, (0, 5), False, 256), (2056, 3584, 272, (5, 0), False, 256), (2304, 3584, 640, (3, 4), False, 256),
    (2052, 3584, 128, (3, 4), False, 256), (2052, 3584, 640, (1, 2), False, 256), (2116, 3584, 256, (1, 2), False, 256),
    (2052, 4096, 640, (0, 0), True, 256), (2052, 4128, 656, (0, 0), True, 256), (2176, 4160, 640, (5, 5), True, 256),
    (2180, 4128, 1296, (0, 5), True, 256), (2056, 4096, 272, (5, 0), True, 256), (2304, 4224, 640, (3, 4), True, 256),
    (2052, 4128, 128, (3, 4), True, 256), (2052, 4128, 640, (1, 2), True, 256), (2116, 4096, 256, (1, 2), True, 256),
    # one to five steps of K and a part of one on three stages; a last tile of 64 columns
    (320, 16000, 128, (0, 0), False, 160), (320, 16032, 256, (5, 5), False, 160), (320, 16000, 384, (0, 5), False, 160),
    (316, 16000, 512, (5, 0), False, 160), (308, 16032, 528, (5, 5), False, 160), (156, 24000, 640, (0, 0), False, 160),
    (300, 16000, 144, (0, 0), False, 160), (300, 16032, 272, (5, 5), False, 160), (292, 16000, 400, (0, 0), False, 160)]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("out", ["f32", "bf16", "fp8"])
def test_exact(L, taken, path, out):
    T.test_exact_on_each_kernel(L, taken, path[:5], out)
    assert {t[:2] for t in taken} == {(T.LARGE, path[5])}


def strided(shape, dtype, ld, first):
    """A view [rows][cols] at column `first` of rows of ld elements, and what lies around it."""
    whole = torch.full((shape[0], ld), 5, dtype=dtype, device="cuda")
    return whole, whole[:, first:first + shape[1]]


def untouched(whole, first, cols):
    assert bool((whole[:, :first] == 5).all()) and bool((whole[:, first + cols:] == 5).all())


# rows that end in the tile's first wavefront, in its second, on and after a strip's end
@pytest.mark.parametrize("M", [2049, 2079, 2175, 2177, 2303])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("asc,bsc", [(0, 0), (5, 5), (1, 2), (3, 4)])
def test_odd_rows_and_strides(L, taken, M, back, asc, bsc):
    odd_rows_and_strides(L, M, 4128 if back else 3584 if asc in (1, 3) else 3552, 384 if asc in (1, 3) else 400, asc, bsc, back)
    assert {t[:2] for t in taken} == {(T.LARGE, 256)}


@pytest.mark.parametrize("M", [289, 303, 317, 319])
@pytest.mark.parametrize("asc,bsc", [(0, 0), (5, 5)])
def test_odd_rows_and_strides_of_160(L, taken, M, asc, bsc):
    odd_rows_and_strides(L, M, 16032, 400, asc, bsc, False)
    assert {t[:2] for t in taken} == {(T.LARGE, 160)}


def odd_rows_and_strides(L, M, F, K, asc, bsc, back):
    nb, n = G.blocks(F), 2 * F if back else F
    g = torch.Generator(device="cuda").manual_seed(M + F + asc)
    A, sa, a = small(g, M, K, int(back), asc)
    B, sb, b = small(g, F if back else 2 * F, K, 0, bsc)
    v = torch.matmul(a, b.t())
    ldt = (M + 3) // 4 * 4 + 12
    whole = {"d": strided((M, n), U8, n + 20, 8), "t": strided((n, M), U8, ldt, 4), "ck": strided((M, 2 * F), U8, 2 * F + 12, 4),
             "exp": strided((M, 2 * nb), U8, 2 * nb + 3, 1), "aux": strided((M, 2 * F), BF, 2 * F + 6, 2)}
    d, t, ck, exp, aux = (whole[k][1] for k in ("d", "t", "ck", "exp", "aux"))
    fmt, f8, top, scale = (1, torch.float8_e5m2, 57344.0, 4.0) if back else (0, torch.float8_e4m3fn, 448.0, 0.25)
    kw = dict(act=L.ACT_RELU, backward=back, d_fmt=fmt, d_scale=torch.full((1,), scale, device="cuda"), D_t=t)
    if back:
        x = torch.tensor([-2.0, -1.0, 1.0, 2.0], device="cuda")[torch.randint(0, 4, (M, 2 * F), generator=g, device="cuda")]
        aux.copy_(x)
        (cg, eg), (cu, eu) = G.save(x[:, :F]), G.save(x[:, F:])
        ck[:, :F], ck[:, F:], exp[:, :nb], exp[:, nb:] = cg, cu, eg, eu
        gate, up = x[:, :F].double(), x[:, F:].double()
        want = torch.cat([v * up * (gate > 0), v * gate.clamp(min=0)], 1)
    else:
        want = (v[:, :F].clamp(min=0) * v[:, F:]).float().double()
    codes = (want * scale).clamp(-top, top).float().to(f8)
    for kept in ("both", "ckpt") if not back else ("bf16", "ckpt"):
        keep = {}
        if kept != "ckpt":
            keep["aux"] = aux
        if kept != "bf16":
            keep["ck"], keep["ck_exp"] = ck, exp
        db = Guarded((2 * F,), F32) if back else None
        if back:
            keep["dbias"] = db.t
        say("gated strides", M, F, K, asc, bsc, back, kept)
        d.fill_(1), t.fill_(1)
        L.fp8_gated_linear(A, int(back), asc, sa, B, 0, bsc, sb, d, **keep, **kw)
        torch.cuda.synchronize()
        assert torch.equal(d.contiguous().view(f8).float(), codes.float())
        assert torch.equal(t, d.t())
        for k, (w, view) in whole.items():
            untouched(w, {"d": 8, "t": 4, "ck": 4, "exp": 1, "aux": 2}[k], view.shape[1])
        if back:
            db.check()
            assert torch.equal(db.t, want.sum(0).float())
            continue
        if kept != "ckpt":
            assert torch.equal(aux, v.float().to(BF))
        for h in (0, 1):
            q, e = G.save(v[:, h * F:(h + 1) * F].float())
            assert torch.equal(ck[:, h * F:(h + 1) * F], q) and torch.equal(exp[:, h * nb:(h + 1) * nb], e)


@pytest.mark.parametrize("M,F,tiles", [(320, 16032, 160), (2052, 3552, 256)])
def test_nan_and_infinity(L, taken, M, F, tiles):
    """A NaN row and a bias of infinity in a large tile: their row, their column, nothing else."""
    K, nb = 256, G.blocks(F)
    g = torch.Generator(device="cuda").manual_seed(1)
    A, sa, a = small(g, M, K, 0, 0)
    B, sb, b = small(g, 2 * F, K, 0, 0)
    v = torch.matmul(a, b.t())
    A[7, 200] = 0x7F
    bias = torch.zeros(2 * F, device="cuda")
    bias[11], bias[F + 50] = float("inf"), float("nan")
    D, amax = torch.empty((M, F), device="cuda"), torch.empty(1, device="cuda")
    ck, exp = torch.empty((M, 2 * F), dtype=U8, device="cuda"), torch.empty((M, 2 * nb), dtype=U8, device="cuda")
    L.fp8_gated_linear(A, 0, 0, sa, B, 0, 0, sb, D, bias=bias, act=L.ACT_RELU, ck=ck, ck_exp=exp, d_amax=amax)
    assert {t[:2] for t in taken} == {(T.LARGE, tiles)}
    want = (v[:, :F].clamp(min=0) * v[:, F:]).float()
    rest = torch.ones((M, F), dtype=torch.bool, device="cuda")
    rest[7], rest[:, 11], rest[:, 50] = False, False, False
    assert torch.equal(D[rest], want[rest])
    assert bool(D[7].isnan().all()) and bool(D[:, 50].isnan().all()) and not bool(D[:, 11].isfinite().any())
    q, e = G.save(v[:, 32:64].float())
    others = torch.arange(M, device="cuda") != 7
    assert torch.equal(exp[others][:, 1], e[others][:, 0]) and torch.equal(ck[others][:, 32:64], q[others])
    assert bool((exp[7] == 127).all()) and bool((exp[:, 0] == 127).all()) and bool((exp[:, nb + 1] == 127).all())
    assert bool(((ck[7] & 0x7F) == 0x7F).all()) and bool(((ck[:, F + 50] & 0x7F) == 0x7F).all())
    assert bool((ck[others][:, 11] == 0x7E).all())
