"""fp8_checkpoint_save / fp8_checkpoint_load against their definition (gated_ref.py),
bit for bit: edge sizes, strides, every exponent, infinities and NaN."""
import pytest
import torch

import gated_ref as G
from gpu_util import Guarded, say

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


def saved(L, x, **kw):
    ck, exp = Guarded(x.shape, U8), Guarded((x.shape[0], G.blocks(x.shape[1])), U8)
    L.fp8_checkpoint_save(x, ck.t, exp.t, **kw)
    torch.cuda.synchronize()
    ck.check(), exp.check()
    return ck.t, exp.t


def check_save(L, x):
    ck, exp = saved(L, x)
    q, e = G.save(x)
    assert torch.equal(exp, e)
    assert torch.equal(ck, q)


SIZES = [(1, 1), (1, 7), (3, 8), (2, 31), (2, 32), (5, 33), (4, 64), (7, 100), (3, 2047), (2, 2048), (2, 2049), (1, 16384), (33, 4095),
         (1531, 2053), (300, 4096), (70000, 9)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sizes(L, size, dtype):
    say("checkpoint", size, dtype)
    g = torch.Generator(device="cuda").manual_seed(size[0] + size[1])
    x = torch.randn(size, generator=g, device="cuda") * torch.exp(2 * torch.randn((size[0], 1), generator=g, device="cuda"))
    x = x.to(dtype)
    check_save(L, x)
    ck, exp = G.save(x)
    y = Guarded(size, dtype)
    L.fp8_checkpoint_load(ck, exp, y.t)
    torch.cuda.synchronize()
    y.check()
    want = G.load(ck, exp)
    assert torch.equal(y.t.double(), want)                       # exact in both types
    err = (want - x.double()).abs()
    top = G.spread(G.block_max(x.double()), size[1])
    # half a step: 2^-4 of a value, or 2^-10 2^-e, and the block's largest is above 224 2^-e
    assert bool((err <= torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 / 224 * top)).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_exponent(L, dtype):
    """Maxima of every exponent, at and beside 1.75 times a power of two; zeros; subnormals."""
    m = torch.tensor([1.0, 1.5, 1.734375, 1.75, 1.7578125, 1.9921875], device="cuda", dtype=torch.float64)
    e = torch.arange(-126, 128, device="cuda", dtype=torch.float64)
    top = (m[:, None] * torch.exp2(e)).reshape(-1)
    top = torch.cat([top, torch.tensor([0.0, 2.0 ** -133, 2.0 ** -127, 2.0 ** -130 * 3], device="cuda", dtype=torch.float64)])
    if dtype == F32:
        top = torch.cat([top, torch.tensor([2.0 ** -149, 448.0, 448.00003051757812, 447.99997], device="cuda", dtype=torch.float64)])
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (2 * torch.rand((top.numel(), 32), generator=g, device="cuda", dtype=torch.float64) - 1) * top[:, None]
    x[:, 5] = top
    check_save(L, x.to(dtype))
    check_save(L, (-x).to(dtype))


def test_infinities_and_nan(L):
    """They stay in their block; the others are untouched."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((6, 130), generator=g, device="cuda")
    x[0, 3], x[1, 40], x[2, 129], x[3, 64], x[3, 65], x[4, 0] = (float(v) for v in ("inf", "-inf", "nan", "nan", "inf", "-nan"))
    for dt in (F32, BF):
        check_save(L, x.to(dt))
        ck, exp = saved(L, x.to(dt))
        y = torch.empty_like(x)
        L.fp8_checkpoint_load(ck, exp, y)
        assert torch.equal(y.isnan(), x.isnan())
        assert float(y[0, 3]) == 448 and float(y[1, 40]) == -448
        assert torch.equal(G.save(x.to(dt))[0][5], ck[5])


def test_every_code_and_byte(L):
    ck = torch.arange(256, dtype=torch.int32, device="cuda").to(U8)
    ck = ck.view(8, 32).repeat(256, 1)                                  # every code in blocks of 32
    exp = torch.arange(256, dtype=torch.int32, device="cuda").to(U8).repeat_interleave(8)[:, None].contiguous()
    want = G.load(ck, exp)
    y = torch.empty((2048, 32), device="cuda")
    L.fp8_checkpoint_load(ck, exp, y)
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y[~want.isnan()], want[~want.isnan()].float())
    assert torch.equal(torch.signbit(y[want == 0]), torch.signbit(want[want == 0]))
    z = torch.empty((2048, 32), device="cuda", dtype=BF)
    L.fp8_checkpoint_load(ck, exp, z)
    normal = want.abs() >= 2.0 ** -126
    assert torch.equal(z[normal], want[normal].float().to(BF)) and torch.equal(z.isnan(), want.isnan())
    assert bool(((z.double() - want).abs() <= 2.0 ** -133)[~normal & ~want.isnan()].all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [70, 96, 333])
def test_strides_and_stream(L, cols, dtype):
    rows, nb, g = 37, G.blocks(cols), torch.Generator(device="cuda").manual_seed(cols)
    big = torch.randn((rows, cols + 11), generator=g, device="cuda").to(dtype)
    x = big[:, 3:3 + cols]
    ck, exp = torch.full((rows, cols + 5), 9, dtype=U8, device="cuda"), torch.full((rows, nb + 3), 9, dtype=U8, device="cuda")
    y = torch.full((rows, cols + 7), 5.0, dtype=dtype, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.fp8_checkpoint_save(x, ck[:, 1:1 + cols], exp[:, 2:2 + nb], stream=s)
    L.fp8_checkpoint_load(ck[:, 1:1 + cols], exp[:, 2:2 + nb], y[:, 1:1 + cols], stream=s)
    s.synchronize()
    q, e = G.save(x)
    assert torch.equal(ck[:, 1:1 + cols], q) and torch.equal(exp[:, 2:2 + nb], e)
    assert torch.equal(y[:, 1:1 + cols].double(), G.load(q, e))
    for t, a, n, v in ((ck, 1, cols, 9), (exp, 2, nb, 9), (y, 1, cols, 5)):
        assert bool((t[:, :a] == v).all()) and bool((t[:, a + n:] == v).all())


def test_types_and_graph(L):
    """float8 views are taken; a captured pair replays on new values."""
    x = torch.randn((65, 300), device="cuda").to(BF)
    ck = torch.empty((65, 300), dtype=torch.float8_e4m3fn, device="cuda")
    exp = torch.empty((65, 10), dtype=torch.float8_e8m0fnu, device="cuda")
    y = torch.empty((65, 300), device="cuda")

    def step():
        L.fp8_checkpoint_save(x, ck, exp)
        L.fp8_checkpoint_load(ck, exp, y)

    step()
    assert torch.equal(ck.float() * G.spread(exp.float(), 300), y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.double(), G.load(*G.save(x))), i


def test_refusals(L):
    x = torch.zeros((4, 64), device="cuda")
    ck, exp = torch.zeros((4, 64), dtype=U8, device="cuda"), torch.zeros((4, 2), dtype=U8, device="cuda")
    for bad in [(x, ck, exp[:, :1]), (x, ck[:, :63], exp), (x[:3], ck, exp), (x, ck.t().contiguous().t(), exp), (x, ck, exp[:1].expand(4, 2))]:
        with pytest.raises(ValueError):
            L.fp8_checkpoint_save(*bad)
        with pytest.raises(ValueError):
            L.fp8_checkpoint_load(bad[1], bad[2], bad[0])
    with pytest.raises(TypeError):
        L.fp8_checkpoint_save(x.half(), ck, exp)
    with pytest.raises(TypeError):
        L.fp8_checkpoint_save(x, ck, exp.float())
    L.fp8_checkpoint_save(x[:0], ck[:0], exp[:0])
    L.fp8_checkpoint_load(ck[:, :0], exp[:, :0], x[:, :0])
