"""fp8_gated_linear, each of its kernels by name: random values with every activation, kept form and
gradient format on the large tiles; exact sums with checkpoints whose powers of two differ from block
to block; exact sums on each of the smaller kernels, which is checked to be the one that was taken."""
import pytest
import torch

import gated_ref as G
import test_gpu_gated as T
from gpu_util import Guarded, say
from test_gpu_gated import FEW, LARGE, TILES, L, taken      # noqa: F401  (fixtures)
from test_gpu_gemm_epilogue import gen
from test_gpu_gemm_epilogue_paths import small

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


# rows a multiple of four, so that D_t's rows start on a dword; a last tile of 32 columns and 4 rows backward,
# of 192 (block scales: 256) columns forward
@pytest.mark.parametrize("asc,bsc,K", [(0, 0, 640), (5, 5, 656), (0, 5, 656), (1, 2, 640), (3, 4, 640)])
@pytest.mark.parametrize("act", [2, 3, 4])
@pytest.mark.parametrize("af", [0, 1])
def test_values_of_large_tiles_backward(L, taken, asc, bsc, K, act, af):
    for j, (kept, out) in enumerate([("bf16", "bf16"), ("ckpt", "e5m2" if af else "e4m3"), ("ckpt", "f32"), ("bf16", "e4m3")]):
        say("gated values", asc, bsc, K, act, af, kept, out)
        T.backward(L, gen(j), 2052, 4128, K, asc, bsc, out, act, kept=kept, p=[BF, F32][j % 2], turned=True, af=af)
    assert set(taken) == {(LARGE, 256, False)}


@pytest.mark.parametrize("asc,bsc,K", [(0, 0, 640), (5, 5, 656), (5, 0, 656), (1, 2, 640), (3, 4, 640)])
@pytest.mark.parametrize("act", [0, 2, 3, 4])
def test_values_of_large_tiles_forward(L, taken, asc, bsc, K, act):
    for j, (kept, out) in enumerate([("ckpt", "e4m3"), ("bf16", "bf16"), ("both", "f32"), ("none", "e5m2")]):
        say("gated values", asc, bsc, K, act, kept, out)
        T.forward(L, gen(j), 2052, 3584 if asc in (1, 3) else 3552, K, asc, bsc, out, act, kept=kept, p=[BF, F32][j % 2],
                  turned=True, bias=j != 1)
    assert set(taken) == {(LARGE, 256, False)}


@pytest.mark.parametrize("asc,bsc,K", [(0, 0, 640), (5, 5, 656)])
@pytest.mark.parametrize("act", [0, 2, 3, 4])
def test_values_of_160_row_tiles(L, taken, asc, bsc, K, act):
    for j, (kept, out) in enumerate([("ckpt", "e4m3"), ("bf16", "bf16"), ("both", "f32")]):
        say("gated values", asc, bsc, K, act, kept, out)
        T.forward(L, gen(j), 316, 16032, K, asc, bsc, out, act, kept=kept, p=[BF, F32][j % 2], turned=True)
    assert set(taken) == {(LARGE, 160, False)}


# rows, outputs, K, scalings, kernel, rows of its tiles, whether K is cut
BACKWARD = [
    (3, 1000, 4112, (0, 0), FEW, 16, False), (13, 264, 4096, (1, 2), FEW, 16, False), (33, 520, 656, (0, 0), TILES, 32, False),
    (64, 512, 8192, (5, 0), TILES, 32, True), (130, 263, 2048, (1, 2), TILES, 32, True), (1037, 1999, 2320, (5, 5), TILES, 64, False),
    (300, 1000, 4096, (3, 3), TILES, 64, True), (1500, 4095, 656, (0, 0), TILES, 128, False), (2048, 4096, 512, (2, 2), TILES, 128, False),
    (2052, 4128, 640, (0, 0), LARGE, 256, False), (2180, 4128, 656, (5, 5), LARGE, 256, False), (2304, 4224, 640, (3, 4), LARGE, 256, False),
    (2052, 4128, 640, (1, 2), LARGE, 256, False)]


@pytest.mark.parametrize("path", BACKWARD)
@pytest.mark.parametrize("out", ["f32", "fp8"])
@pytest.mark.parametrize("af", [0, 1])
def test_every_block_has_a_power_of_its_own(L, taken, path, out, af):
    """A checkpoint read with powers of two that differ by row, block of 32 columns and half: up to 2^3
    times the small integers whose sums are exact, so another row's, block's or half's byte shows."""
    M, F, K, (asc, bsc) = path[:4]
    nb = G.blocks(F)
    g = torch.Generator(device="cuda").manual_seed(M + F + K + af)
    A, sa, a = small(g, M, K, af, asc)
    B, sb, b = small(g, F, K, 0, bsc)
    v = torch.matmul(a, b.t())
    power = torch.randint(0, 4, (M, 2 * nb), generator=g, device="cuda")
    x = torch.tensor([-2.0, -1.0, 1.0, 2.0], device="cuda")[torch.randint(0, 4, (M, 2 * F), generator=g, device="cuda")]
    for h in (0, 1):
        half = x[:, h * F:(h + 1) * F]
        half[:, ::32] = 2.0                           # every block has its largest value
        half.mul_(G.spread(torch.exp2(power[:, h * nb:(h + 1) * nb].float()), F))
    (cg, eg), (cu, eu) = G.save(x[:, :F]), G.save(x[:, F:])
    exp = torch.cat([eg, eu], 1)
    assert torch.equal(exp.int() - exp.int().amin(), power.int()), "the bytes are the powers"
    gate, up = x[:, :F].double(), x[:, F:].double()
    want = torch.cat([v * up * (gate > 0), v * gate.clamp(min=0)], 1)
    assert float(want.abs().sum(0).max()) < 2 ** 24, "column sums are exact"
    D, db, amax = Guarded((M, 2 * F), U8 if out == "fp8" else F32), Guarded((2 * F,), F32), Guarded((1,), F32)
    kw, scale, f8 = {}, 1.0, torch.float8_e5m2
    if out == "fp8":
        scale = 0.25
        D_t = Guarded((2 * F, M), U8)
        kw = dict(d_fmt=L.E5M2, d_scale=torch.full((1,), scale, device="cuda"), D_t=D_t.t)
    say("gated powers", path, out, af)
    L.fp8_gated_linear(A, af, asc, sa, B, 0, bsc, sb, D.t, act=L.ACT_RELU, backward=True, ck=torch.cat([cg, cu], 1), ck_exp=exp,
                       dbias=db.t, d_amax=amax.t, **kw)
    torch.cuda.synchronize()
    D.check(), db.check(), amax.check()
    if out == "fp8":
        D_t.check()
        assert torch.equal(D.t.view(f8).float(), (want * scale).clamp(-57344, 57344).float().to(f8).float())
        assert torch.equal(D_t.t, D.t.t())
    else:
        assert torch.equal(D.t, want.float())
    assert torch.equal(db.t, want.sum(0).float())
    assert float(amax.t) == float(want.abs().max())
    assert taken == [path[4:7]]


# rows, outputs, K, scalings, direction, and (kernel, rows of its tiles, whether K is cut): what a call that
# keeps or reads a checkpoint takes, and one with BF16 (the few-row kernel writes no checkpoints).  Tiles are named
# where they are the faster ones, not where a width or an alignment keeps a call off the large kernels.
PATHS = [
    (3, 1000, 4112, (0, 0), False, (TILES, 32, True), (FEW, 16, False)), (16, 520, 2064, (5, 5), False, (TILES, 32, False), (FEW, 16, False)),
    (7, 330, 2048, (1, 2), False, (TILES, 32, True), (FEW, 16, False)), (7, 328, 2048, (1, 1), False, (TILES, 32, True), (FEW, 16, False)),
    (16, 136, 1024, (3, 4), False, (TILES, 32, False), (FEW, 16, False)), (33, 260, 656, (0, 0), False, (TILES, 32, False), None),
    (64, 256, 8192, (5, 0), False, (TILES, 32, True), None), (130, 136, 2048, (1, 2), False, (TILES, 32, True), None),
    (130, 132, 2048, (3, 4), False, (TILES, 32, True), None), (1037, 999, 2320, (5, 5), False, (TILES, 64, False), None),
    (1037, 1000, 2304, (1, 2), False, (TILES, 64, False), None), (1500, 1000, 384, (3, 4), False, (TILES, 64, False), None),
    (300, 500, 4096, (1, 2), False, (TILES, 64, True), None), (300, 500, 4096, (3, 3), False, (TILES, 64, True), None),
    (1100, 2047, 656, (0, 0), False, (TILES, 128, False), None), (2048, 2048, 512, (2, 2), False, (TILES, 128, False), None),
    (2048, 2048, 512, (4, 3), False, (TILES, 128, False), None),
    (3, 1000, 4112, (0, 0), True, (FEW, 16, False), None), (13, 264, 4096, (1, 2), True, (FEW, 16, False), None),
    (33, 520, 656, (0, 0), True, (TILES, 32, False), None), (64, 512, 8192, (5, 0), True, (TILES, 32, True), None),
    (130, 264, 2048, (1, 1), True, (TILES, 32, True), None), (1037, 1999, 2320, (5, 5), True, (TILES, 64, False), None),
    (1037, 1999, 2304, (1, 2), True, (TILES, 64, False), None), (300, 1000, 4096, (3, 3), True, (TILES, 64, True), None),
    (1500, 4095, 656, (0, 0), True, (TILES, 128, False), None), (2048, 4096, 512, (2, 2), True, (TILES, 128, False), None)]


@pytest.mark.parametrize("path", PATHS)
def test_exact_on_the_named_kernel(L, taken, path):
    *call, ckpt, bf16 = path
    T.test_exact_on_each_kernel(L, taken, call, ["f32", "bf16", "fp8"][PATHS.index(path) % 3])
    assert taken == [ckpt, bf16 or ckpt]
