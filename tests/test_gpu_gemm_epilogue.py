"""fp8_scaled_gemm_ep against its 64-bit form (block_ref.py): every scaling,
format pair, output type, activation and direction, edge sizes, strides, K parts
and repeated calls."""
import pytest
import torch

import block_ref as R
from gpu_util import Guarded, say

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def operand(g, rows, K, fmt, scaling, std=1.0, ld=None):
    """Codes [rows][K] (row stride ld) and inverse scales of N(0, std) values."""
    x = rand(g, (rows, K), std)
    nkb, nrb = -(-K // 128), -(-rows // 128)
    if scaling == 0:
        s = x.abs().amax().reshape(1) / R.FMAX[fmt]
        w = s
    elif scaling == 5:
        s = x.abs().amax(1) / R.FMAX[fmt]
        w = s[:, None]
    else:
        pad = torch.zeros((nrb * 128, nkb * 128), device="cuda")
        pad[:rows, :K] = x
        seg = scaling in (1, 3)
        s = (pad.view(nrb * 128, nkb, 128).abs().amax(2).t()[:, :rows] if seg
             else pad.view(nrb, 128, nkb, 128).abs().amax((1, 3)).t()) / R.FMAX[fmt]
        if scaling in (3, 4):
            s = torch.exp2(torch.ceil(torch.log2(s)))
        s = s.contiguous()
        w = s.t().repeat_interleave(128, 1)
        w = w if seg else w.repeat_interleave(128, 0)[:rows]
    q = (x / w).clamp(-R.FMAX[fmt], R.FMAX[fmt]).to(R.F8[fmt]).view(torch.uint8)
    if ld is not None:
        big = torch.randint(0, 256, (rows, ld), generator=g, device="cuda", dtype=torch.uint8)
        big[:, :K] = q
        q = big[:, :K]
    return q, s.float()


def call(L, g, M, N, K, af, bf, asc, bsc, out, act, backward, *, bias=True, residual=False, aux=True, p=F32, turned=False,
         res_dtype=BF, res_scale=1.0, lda=None, ldb=None):
    A, sa = operand(g, M, K, af, asc, 1.0, lda)
    B, sb = operand(g, N, K, bf, bsc, 0.5 / max(1, K) ** 0.5, ldb)
    v, E = R.product(A, af, asc, sa, B, bf, bsc, sb)
    dt = {"bf16": BF, "f32": F32, "e4m3": torch.uint8, "e5m2": torch.uint8}[out]
    D = Guarded((M, N), dt)
    kw = dict(act=act, backward=backward)
    fmt = {"e4m3": 0, "e5m2": 1}.get(out)
    amax = Guarded((1,), F32)
    kw["d_amax"] = amax.t
    D_t = None
    if fmt is not None:
        kw["d_fmt"], kw["d_scale"] = fmt, torch.tensor([60.0 if fmt == 0 else 4000.0], device="cuda")
        if turned:
            D_t = Guarded((N, M), torch.uint8)
            kw["D_t"] = D_t.t
    b = r = x = db = None
    if backward:
        if act:
            x = rand(g, (M, N), 1.5, BF)
            kw["aux"] = x
        if bias:
            db = Guarded((N,), p)
            kw["dbias"] = db.t
    else:
        if bias:
            b = rand(g, (N,), 0.5, p)
            kw["bias"] = b
        if residual:
            r = rand(g, (M, N), 1.0, res_dtype)
            kw["residual"], kw["res_scale"] = r, res_scale
        if aux:
            x = Guarded((M, N), BF)
            kw["aux"] = x.t
    L.fp8_scaled_gemm_ep(A, af, asc, sa, B, bf, bsc, sb, D.t, **kw)
    torch.cuda.synchronize()
    D.check(), amax.check()
    if backward:
        o, Eo = R.linear_bwd(v, E, x, act)
        if db is not None:
            db.check()
            R.close(db.t, o.sum(0), Eo.sum(0) + (R.C + M * 2.0 ** -24) * o.abs().sum(0))
    else:
        (u, Eu), (o, Eo) = R.linear_fwd(v, E, b, act, r, res_scale)
        if aux:
            x.check()
            R.close(x.t, u, Eu)
    if fmt is None:
        R.close(D.t, o, Eo)
    else:
        s = float(kw["d_scale"])
        R.close8(D.t, fmt, o * s, Eo * s)
        if D_t is not None:
            D_t.check()
            assert torch.equal(D_t.t, D.t.t())
    R.close(amax.t, o.abs().max().reshape(1), Eo.max() + (2.0 ** -8 if out == "bf16" else 0) * o.abs().max())


SCALINGS = [(0, 0), (5, 5), (5, 0), (0, 5), (1, 2), (1, 1), (2, 1), (2, 2), (3, 4), (3, 3), (4, 3), (1, 4), (0, 2), (1, 0),
            (0, 4), (3, 0)]


@pytest.mark.parametrize("asc,bsc", SCALINGS)
@pytest.mark.parametrize("backward", [False, True])
def test_scalings(L, asc, bsc, backward):
    i = SCALINGS.index((asc, bsc))
    M, N, K = [(200, 264, 384), (130, 129, 256), (33, 520, 640)][i % 3]
    out = ["bf16", "f32", "e5m2" if backward else "e4m3"][i % 3]
    say("ep scaling", asc, bsc, backward, M, N, K, out)
    call(L, gen(i), M, N, K, int(backward), 0, asc, bsc, out, 1 + i % 4, backward, turned=i % 2 == 0, p=[BF, F32][i % 2])


@pytest.mark.parametrize("af,bf", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("asc,bsc", [(0, 0), (1, 2), (3, 4)])
def test_formats(L, af, bf, asc, bsc):
    say("ep formats", af, bf, asc, bsc)
    call(L, gen(5), 140, 200, 256, af, bf, asc, bsc, "bf16", 4, False)
    call(L, gen(6), 140, 200, 256, af, bf, asc, bsc, "e4m3", 4, False, turned=True)


SIZES = [(1, 1, 16), (1, 4096, 2048), (2, 640, 4096), (3, 17, 48), (15, 100, 128), (16, 2048, 1024), (17, 384, 4096),
         (31, 1999, 512), (32, 33, 2064), (33, 4097, 1024), (64, 512, 8192), (65, 130, 272), (100, 3000, 4096), (127, 128, 144),
         (128, 127, 1024), (129, 255, 2048), (257, 513, 112), (300, 1000, 4096), (520, 776, 1536), (1037, 1999, 2304)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("blocks", [False, True])
def test_sizes(L, size, backward, blocks):
    M, N, K = size
    i = SIZES.index(size)
    if blocks:
        K = -(-K // 128) * 128
    asc, bsc = ((1, 2), (3, 4))[i % 2] if blocks else ((0, 0), (5, 5))[i % 2]
    out = ["bf16", "f32", "e4m3"][(i + backward) % 3]
    say("ep size", M, N, K, backward, asc, bsc, out)
    call(L, gen(M + N), M, N, K, int(backward), 0, asc, bsc, out, [3, 0, 2, 4, 1][i % 5], backward, residual=i % 2 == 0,
         turned=i % 3 != 0, aux=i % 4 != 0, res_scale=0.5, res_dtype=F32 if i % 2 and out != "e4m3" else BF)


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("backward", [False, True])
def test_large(L, blocks, out, backward):
    """Sizes of the large tiles, with edges."""
    M, N, K = 2050, 4104, 640
    asc, bsc = (1, 2) if blocks else (0, 0)
    say("ep large", blocks, out, backward)
    call(L, gen(1), M, N, K, int(backward), 0, asc, bsc, out, 3, backward, turned=True)
    if not blocks:
        call(L, gen(2), 4096, 2048, 656, int(backward), 0, 5, 5, out, 4, backward, turned=False)
        call(L, gen(3), 2048, 4096, 512, int(backward), 0, 3, 4, out, 4, backward, turned=True)


def test_activations(L):
    """Every activation and its slope over a wide range of pre-activations."""
    for act in range(5):
        for backward in (False, True):
            call(L, gen(act), 70, 300, 256, 0, 0, 0, 0, "f32", act, backward)
    A = torch.full((1, 128), 0x38, dtype=torch.uint8, device="cuda")   # 1.0
    B = torch.zeros((16, 128), dtype=torch.uint8, device="cuda")
    B[:, 0] = 0x38                                                     # v = 1
    one = torch.ones(1, device="cuda")
    aux = torch.tensor([[-1e30, -3e4, -100, -30, -8, -1e-3, -0.0, 0.0, 1e-30, 1e-3, 1, 8, 30, 100, 3e4, 1e30]],
                       device="cuda").to(BF)
    for act in range(1, 5):
        D = torch.empty((1, 16), device="cuda")
        L.fp8_scaled_gemm_ep(A, 0, 0, one, B, 0, 0, one, D, act=act, aux=aux, backward=True)
        want = R.slope_of(aux.double(), act)
        want = torch.where(want.isnan(), (aux.double() > 0).double(), want)
        R.close(D, want, R.C * torch.ones_like(want))
        bias = aux[0].float() - 1
        L.fp8_scaled_gemm_ep(A, 0, 0, one, B, 0, 0, one, D, act=act, bias=bias)
        u = (bias + 1).double()[None]
        want = R.act_of(u, act)
        R.close(D, want, R.C * (1 + u.abs()) * (u.abs() < 1e3) + 2 * R.C * want.abs())


def test_strides_in_place_residual_and_stream(L):
    M, N, K = 77, 203, 384
    g = gen(3)
    A, sa = operand(g, M, K, 0, 5, 1.0, K + 32)
    B, sb = operand(g, N, K, 0, 5, 0.03, K + 16)
    v, E = R.product(A, 0, 5, sa, B, 0, 5, sb)
    big = rand(g, (M, N + 9), 1.0, F32)
    stream = big[:, 4:4 + N]
    edge = big.clone()
    aux = torch.full((M, N + 3), 3.0, dtype=BF, device="cuda")
    (u, Eu), (o, Eo) = R.linear_fwd(v, E, None, 4, stream, 0.5)
    s = torch.cuda.Stream()
    ws = torch.empty(L.fp8_scaled_gemm_ep_workspace(M, N, K, 5, 5), dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    L.fp8_scaled_gemm_ep(A, 0, 5, sa, B, 0, 5, sb, stream, act=4, aux=aux[:, 1:1 + N], residual=stream, res_scale=0.5,
                         workspace=ws, stream=s)
    s.synchronize()
    R.close(stream, o, Eo)
    R.close(aux[:, 1:1 + N], u, Eu)
    assert torch.equal(big[:, :4], edge[:, :4]) and torch.equal(big[:, 4 + N:], edge[:, 4 + N:])
    assert bool((aux[:, 0] == 3).all()) and bool((aux[:, 1 + N:] == 3).all())


def test_no_k_no_rows(L):
    one = torch.ones(1, device="cuda")
    A = torch.empty((5, 0), dtype=torch.uint8, device="cuda")
    B = torch.empty((9, 0), dtype=torch.uint8, device="cuda")
    bias, D = torch.arange(9.0, device="cuda"), torch.full((5, 9), 7.0, device="cuda")
    L.fp8_scaled_gemm_ep(A, 0, 0, one, B, 0, 0, one, D, bias=bias, act=1)
    assert torch.equal(D, bias.expand(5, 9))
    db = torch.full((9,), 7.0, device="cuda")
    L.fp8_scaled_gemm_ep(torch.empty((0, 128), dtype=torch.uint8, device="cuda"), 0, 0, one,
                         torch.zeros((9, 128), dtype=torch.uint8, device="cuda"), 0, 0, one,
                         torch.empty((0, 9), device="cuda"), backward=True, dbias=db)
    assert bool((db == 0).all())


def test_nan_stays_in_its_row_and_column(L):
    M, N, K = 40, 60, 256
    g = gen(1)
    A, sa = operand(g, M, K, 0, 0)
    B, sb = operand(g, N, K, 0, 0)
    A[7, 200] = 0x7F
    bias = torch.zeros(N, device="cuda")
    bias[11] = float("inf")
    D = torch.empty((M, N), device="cuda")
    L.fp8_scaled_gemm_ep(A, 0, 0, sa, B, 0, 0, sb, D, bias=bias, act=4)
    bad = D.isnan()
    assert bool(bad[7].all()) and not bool(bad[torch.arange(M, device="cuda") != 7].any())
    assert bool(D[torch.arange(M, device="cuda") != 7][:, 11].isinf().all())


@pytest.mark.parametrize("size", [(4, 640, 4096), (300, 520, 1024)])
def test_repeatable_and_graph(L, size):
    M, N, K = size
    g = gen(2)
    A, sa = operand(g, M, K, 1, 0)
    B, sb = operand(g, N, K, 0, 0)
    aux = rand(g, (M, N), 1.0, BF)
    D, db = torch.empty((M, N), dtype=BF, device="cuda"), torch.empty(N, device="cuda")
    ws = torch.empty(L.fp8_scaled_gemm_ep_workspace(M, N, K, 0, 0), dtype=torch.uint8, device="cuda")
    amax = torch.empty(1, device="cuda")

    def step():
        L.fp8_scaled_gemm_ep(A, 1, 0, sa, B, 0, 0, sb, D, act=3, aux=aux, backward=True, dbias=db, d_amax=amax, workspace=ws)
        return [t.clone() for t in (D, db, amax)]

    first = step()
    for a, b in zip(first, step()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(4):
        aux.normal_()
        ws.random_(0, 255)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i
