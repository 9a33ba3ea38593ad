"""fp8_gated_linear against its 64-bit form (gated_ref.py): both directions, every
scaling, activation and output type, g and u kept in BF16 and as a checkpoint, edge
sizes, strides, K parts, exact values on each kernel, differences, repeated calls."""
import ctypes as C

import pytest
import torch

import block_ref as R
import gated_ref as G
from gpu_util import Guarded, say
from test_gpu_gemm_epilogue import gen, operand, rand
from test_gpu_gemm_epilogue_paths import small

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
DTYPE = {"bf16": BF, "f32": F32, "e4m3": U8, "e5m2": U8}


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


@pytest.fixture
def taken(L, monkeypatch):
    """The kernels that the calls of a test have taken."""
    call, seen = L._L.fp8_gated_linear, []

    def spy(gemm, ep, stream):
        plan = L.EpPlan()
        assert L._L.fp8_gated_linear_plan(gemm, ep, C.byref(plan)) == 0
        seen.append((plan.kernel, plan.tile_rows, plan.k_parts > 1))
        return call(gemm, ep, stream)

    monkeypatch.setattr(L._L, "fp8_gated_linear", spy)
    return seen


def outputs(shape, out, turned, kw):
    D, amax = Guarded(shape, DTYPE[out]), Guarded((1,), F32)
    kw["d_amax"], D_t = amax.t, None
    fmt = {"e4m3": 0, "e5m2": 1}.get(out)
    if fmt is not None:
        kw["d_fmt"], kw["d_scale"] = fmt, torch.tensor([60.0 if fmt == 0 else 4000.0], device="cuda")
        if turned:
            D_t = Guarded(shape[::-1], U8)
            kw["D_t"] = D_t.t
    return D, D_t, amax, fmt


def check_outputs(D, D_t, amax, fmt, kw, out, o, Eo):
    D.check(), amax.check()
    if fmt is None:
        R.close(D.t, o, Eo)
    else:
        s = float(kw["d_scale"])
        R.close8(D.t, fmt, o * s, Eo * s)
        if D_t is not None:
            D_t.check()
            assert torch.equal(D_t.t, D.t.t())
    R.close(amax.t, o.abs().max().reshape(1), Eo.max() + (2.0 ** -8 if out == "bf16" else 0) * o.abs().max())


def forward(L, g, M, F, K, asc, bsc, out, act, *, bias=True, kept="ckpt", p=F32, turned=False):
    A, sa = operand(g, M, K, 0, asc)
    B, sb = operand(g, 2 * F, K, 0, bsc, 1.5 / max(1, K) ** 0.5)
    kw = dict(act=act)
    D, D_t, amax, fmt = outputs((M, F), out, turned, kw)
    b = rand(g, (2 * F,), 0.5, p) if bias else None
    aux = Guarded((M, 2 * F), BF) if kept in ("bf16", "both") else None
    ck, exp = (Guarded((M, 2 * F), U8), Guarded((M, 2 * G.blocks(F)), U8)) if kept in ("ckpt", "both") else (None, None)
    if aux:
        kw["aux"] = aux.t
    if ck:
        kw["ck"], kw["ck_exp"] = ck.t, exp.t
    L.fp8_gated_linear(A, 0, asc, sa, B, 0, bsc, sb, D.t, bias=b, **kw)
    torch.cuda.synchronize()
    v, E = R.product(A, 0, asc, sa, B, 0, bsc, sb)
    (x, Ex), (o, Eo) = G.forward(v, E, b, act)
    if aux:
        aux.check()
        R.close(aux.t, x, Ex)
    if ck:
        ck.check(), exp.check()
        nb = G.blocks(F)
        G.close_checkpoint(ck.t[:, :F], exp.t[:, :nb], x[:, :F], Ex[:, :F])
        G.close_checkpoint(ck.t[:, F:], exp.t[:, nb:], x[:, F:], Ex[:, F:])
    check_outputs(D, D_t, amax, fmt, kw, out, o, Eo)


def backward(L, g, M, F, K, asc, bsc, out, act, *, bias=True, kept="ckpt", p=F32, turned=False, af=1):
    A, sa = operand(g, M, K, af, asc)
    B, sb = operand(g, F, K, 0, bsc, 0.5 / max(1, K) ** 0.5)
    kw = dict(act=act)
    D, D_t, amax, fmt = outputs((M, 2 * F), out, turned, kw)
    db = Guarded((2 * F,), p) if bias else None
    if db:
        kw["dbias"] = db.t
    x = rand(g, (M, 2 * F), 1.5)
    if kept == "bf16":
        kw["aux"] = x = x.to(BF)
    else:
        (cg, eg), (cu, eu) = G.save(x[:, :F]), G.save(x[:, F:])
        kw["ck"], kw["ck_exp"] = torch.cat([cg, cu], 1), torch.cat([eg, eu], 1)
        x = torch.cat([G.load(cg, eg), G.load(cu, eu)], 1)
    L.fp8_gated_linear(A, af, asc, sa, B, 0, bsc, sb, D.t, backward=True, **kw)
    torch.cuda.synchronize()
    v, E = R.product(A, af, asc, sa, B, 0, bsc, sb)
    o, Eo = G.backward(v, E, x, act)
    check_outputs(D, D_t, amax, fmt, kw, out, o, Eo)
    if db:
        db.check()
        R.close(db.t, o.sum(0), Eo.sum(0) + (R.C + M * 2.0 ** -24) * o.abs().sum(0))


WAY = {False: forward, True: backward}
SCALINGS = [(0, 0), (5, 5), (5, 0), (0, 5), (1, 2), (1, 1), (2, 1), (2, 2), (3, 4), (3, 3), (4, 3), (1, 4), (0, 2), (1, 0), (0, 4), (3, 0)]


@pytest.mark.parametrize("asc,bsc", SCALINGS)
@pytest.mark.parametrize("back", [False, True])
def test_scalings(L, asc, bsc, back):
    i = SCALINGS.index((asc, bsc))
    for j, (M, F, K) in enumerate([(200, 264, 384), (130, 129, 256), (33, 520, 640), (7, 208, 512)]):
        out = ["bf16", "f32", "e5m2" if back else "e4m3"][(i + j) % 3]
        say("gated scaling", asc, bsc, back, M, F, K, out)
        WAY[back](L, gen(i), M, F, K, asc, bsc, out, 1 + (i + j) % 4, turned=(i + j) % 2 == 0, p=[BF, F32][i % 2],
                  kept=["ckpt", "bf16"][(i + j) % 2])


SIZES = [(1, 1, 16), (1, 4096, 2048), (2, 640, 4096), (3, 17, 48), (15, 100, 128), (16, 2048, 1024), (17, 384, 4096),
         (31, 1999, 512), (32, 33, 2064), (33, 4097, 1024), (64, 512, 8192), (65, 130, 272), (100, 2000, 4096), (127, 64, 144),
         (128, 63, 1024), (129, 255, 2048), (257, 513, 112), (300, 1000, 4096), (520, 776, 1536), (777, 1999, 2304)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("blocks", [False, True])
def test_sizes(L, size, back, blocks):
    M, F, K = size
    i = SIZES.index(size)
    if blocks:
        K = -(-K // 128) * 128
    asc, bsc = ((1, 2), (3, 4))[i % 2] if blocks else ((0, 0), (5, 5))[i % 2]
    for j, kept in enumerate(["ckpt", "bf16"] if back else ["ckpt", "both", "none"]):
        out = ["bf16", "f32", "e4m3"][(i + j + back) % 3]
        say("gated size", M, F, K, back, asc, bsc, out, kept)
        WAY[back](L, gen(M + F), M, F, K, asc, bsc, out, [4, 0, 2, 3, 1][(i + j) % 5], kept=kept, bias=(i + j) % 2 == 0,
                  turned=i % 3 != 0)


@pytest.mark.parametrize("size", [(2050, 4104, 640), (1100, 4096, 656), (2048, 2048, 512)])
@pytest.mark.parametrize("asc,bsc", [(0, 0), (5, 5), (1, 2), (3, 4)])
@pytest.mark.parametrize("back", [False, True])
def test_large(L, size, asc, bsc, back):
    M, F, K = size
    if asc in (1, 3):
        K = K // 128 * 128
    for j, (kept, out) in enumerate([("ckpt", "e4m3"), ("bf16", "bf16"), ("ckpt", "f32")]):
        say("gated large", size, asc, bsc, back, kept, out)
        more = dict(af=j % 2) if back else {}
        WAY[back](L, gen(j), M, F, K, asc, bsc, out, 4 - j, kept=kept, turned=True, **more)


@pytest.mark.parametrize("af", [0, 1])
@pytest.mark.parametrize("asc,bsc", [(0, 0), (1, 2), (1, 1), (3, 4)])
def test_gradient_formats(L, af, asc, bsc):
    for M in (9, 140, 600):
        backward(L, gen(5), M, 200, 256, asc, bsc, "bf16", 4, af=af)
        backward(L, gen(6), M, 200, 256, asc, bsc, "e5m2", 4, af=af, turned=True)


@pytest.mark.parametrize("back", [False, True])
def test_activations(L, back):
    for act in range(5):
        for M in (5, 70):
            WAY[back](L, gen(act), M, 300, 256, 0, 0, "f32", act)


def one_row(F):
    """A product whose every value is 1."""
    A = torch.full((1, 128), 0x38, dtype=U8, device="cuda")   # 1.0
    B = torch.zeros((F, 128), dtype=U8, device="cuda")
    B[:, 0] = 0x38
    return A, B


def test_far_activations(L):
    """Pre-activations far out: slopes reach their limits, nothing turns into NaN."""
    far = [-1e30, -3e4, -100, -30, -8, -1e-3, -0.0, 0.0, 1e-30, 1e-3, 1, 8, 30, 100, 3e4, 1e30]
    one, F = torch.ones(1, device="cuda"), len(far)
    A, B = one_row(F)
    aux = torch.cat([torch.tensor([far], device="cuda"), torch.full((1, F), 2.0, device="cuda")], 1).to(BF)
    for act in range(1, 5):
        D = torch.empty((1, 2 * F), device="cuda")
        L.fp8_gated_linear(A, 0, 0, one, B, 0, 0, one, D, act=act, aux=aux, backward=True)
        g = aux[:, :F].double()
        s = R.slope_of(g, act)
        s = torch.where(s.isnan(), (g > 0).double(), s)
        a = R.act_of(g, act)
        a = torch.where(a.isnan(), g.clamp(min=0), a)
        R.close(D[:, :F], 2 * s, 2 * R.C * torch.ones_like(s))
        R.close(D[:, F:], a, R.C * (1 + g.abs()) * (g.abs() < 1e3) + 2 * R.C * a.abs())


def test_differences(L):
    """dbias is the derivative of sum(h * dy) by the biases, as the forward call has it."""
    M, F, K = 40, 24, 128
    g = gen(11)
    A, sa = operand(g, M, K, 0, 5)
    B, sb = operand(g, 2 * F, K, 0, 5, 0.1)
    bias = rand(g, (2 * F,), 0.5)
    dy = torch.tensor([-2.0, -1.0, 0.0, 1.0, 2.0], device="cuda")[torch.randint(0, 5, (M, F), generator=g, device="cuda")]
    codes = dy.to(torch.float8_e5m2).view(U8)
    pad = torch.zeros((M, 128), dtype=U8, device="cuda")
    pad[:, :F] = codes
    eye = torch.zeros((F, 128), dtype=U8, device="cuda")
    eye[torch.arange(F), torch.arange(F)] = 0x38                    # the next linear is the identity
    one = torch.ones(1, device="cuda")
    aux = torch.empty((M, 2 * F), dtype=BF, device="cuda")

    def h(b, act, keep=None):
        D = torch.empty((M, F), device="cuda")
        L.fp8_gated_linear(A, 0, 5, sa, B, 0, 5, sb, D, act=act, bias=b, aux=keep)
        return D.double()

    for act in (0, 2, 3, 4):
        h(bias, act, aux)
        D, db = torch.empty((M, 2 * F), device="cuda"), torch.empty(2 * F, device="cuda")
        L.fp8_gated_linear(pad, 1, 0, one, eye, 0, 0, one, D, act=act, aux=aux, backward=True, dbias=db)
        step = 2.0 ** -6
        for k in (0, 7, 23, 24, 30, 47):
            d = torch.zeros_like(bias)
            d[k] = step
            f = k % F
            slope = (((h(bias + d, act) - h(bias - d, act))[:, f] * dy[:, f]).sum() / (2 * step)).item()
            # the third derivative of act(g) u is below 4 (1 + |u|), the forward values' rounding is
            # 2^-24 of them, and g and u were kept to 2^-8
            x = aux.double()
            size = ((1 + x[:, f].abs()) * (1 + x[:, F + f].abs()) * dy[:, f].abs()).sum().item()
            assert abs(slope - db[k].item()) <= size * (4 * step ** 2 / 6 + 2.0 ** -22 / step + 2 * 2.0 ** -8), (act, k)


def test_no_k_no_rows_no_outputs(L):
    one = torch.ones(1, device="cuda")
    for scalings in [(0, 0), (5, 5), (1, 2), (3, 4), (0, 2)]:
        for M in (5, 40, 300):
            F = 72
            A, B = torch.empty((M, 0), dtype=U8, device="cuda"), torch.empty((2 * F, 0), dtype=U8, device="cuda")
            bias = torch.randn(2 * F, generator=gen(M), device="cuda")
            D, aux = Guarded((M, F), F32), Guarded((M, 2 * F), BF)
            ck, exp = Guarded((M, 2 * F), U8), Guarded((M, 2 * 3), U8)
            L.fp8_gated_linear(A, 0, scalings[0], None, B, 0, scalings[1], None, D.t, act=L.ACT_RELU, bias=bias, aux=aux.t,
                               ck=ck.t, ck_exp=exp.t)
            torch.cuda.synchronize()
            for t in (D, aux, ck, exp):
                t.check()
            assert torch.equal(D.t, (bias[:F].clamp(min=0) * bias[F:]).expand(M, F))
            assert torch.equal(aux.t, bias.to(BF).expand(M, 2 * F))
            for half in (0, 1):
                q, e = G.save(bias[half * F:(half + 1) * F][None])
                assert torch.equal(ck.t[:, half * F:(half + 1) * F], q.expand(M, F))
                assert torch.equal(exp.t[:, half * 3:half * 3 + 3], e.expand(M, 3))
            db = torch.full((2 * F,), 7.0, device="cuda")
            W = Guarded((M, 2 * F), F32)
            L.fp8_gated_linear(A, 1, scalings[0], None, B[:F], 0, scalings[1], None, W.t, ck=ck.t, ck_exp=exp.t, backward=True, dbias=db)
            torch.cuda.synchronize()
            W.check()
            assert bool((W.t == 0).all()) and bool((db == 0).all())
    none = torch.empty((0, 128), dtype=U8, device="cuda")
    db = torch.full((18,), 7.0, device="cuda")
    L.fp8_gated_linear(none, 1, 0, one, torch.zeros((9, 128), dtype=U8, device="cuda"), 0, 0, one, torch.empty((0, 18), device="cuda"),
                       aux=torch.empty((0, 18), dtype=BF, device="cuda"), backward=True, dbias=db)
    assert bool((db == 0).all())
    amax = torch.full((1,), 7.0, device="cuda")
    L.fp8_gated_linear(torch.zeros((4, 128), dtype=U8, device="cuda"), 0, 0, one, none, 0, 0, one, torch.empty((4, 0), device="cuda"), d_amax=amax)
    assert float(amax) == 0


def test_nan_stays_in_its_row_and_column(L):
    for M in (9, 40, 300):
        F, K, g = 70, 256, gen(1)
        A, sa = operand(g, M, K, 0, 0)
        B, sb = operand(g, 2 * F, K, 0, 0)
        A[7, 200] = 0x7F
        bias = torch.zeros(2 * F, device="cuda")
        bias[11], bias[F + 50] = float("inf"), float("nan")
        D = torch.empty((M, F), device="cuda")
        ck, exp = torch.empty((M, 2 * F), dtype=U8, device="cuda"), torch.empty((M, 6), dtype=U8, device="cuda")
        L.fp8_gated_linear(A, 0, 0, sa, B, 0, 0, sb, D, bias=bias, act=L.ACT_SILU, ck=ck, ck_exp=exp)
        others = torch.arange(M, device="cuda") != 7
        bad = D.isnan()
        assert bool(bad[7].all()) and bool(bad[:, 50].all())
        bad[:, 50] = False
        assert not bool(bad[others].any()) and bool(D[others][:, 11].isinf().all())
        # blocks that hold one have the power 0, the others their own
        assert bool((exp[7] == 127).all()) and bool((exp[:, 0] == 127).all()) and bool((exp[:, 4] == 127).all())
        q, e = G.save((R.product(A, 0, 0, sa, B, 0, 0, sb)[0])[others][:, 32:64])
        assert bool(((exp[others][:, 1].int() - e[:, 0].int()).abs() <= 1).all())
        assert bool(((ck[7] & 0x7F) == 0x7F).all()) and bool(((ck[:, F + 50] & 0x7F) == 0x7F).all())
        assert bool((ck[others][:, 11] == 0x7E).all())                           # 448


@pytest.mark.parametrize("kept", ["bf16", "ckpt"])
@pytest.mark.parametrize("M", [5, 77])
def test_strides_and_stream(L, M, kept):
    F, K, nb = 203, 384, 7
    g = gen(3)
    s = torch.cuda.Stream()
    A, sa = operand(g, M, K, 0, 5, 1.0, K + 32)
    B, sb = operand(g, 2 * F, K, 0, 5, 0.08, K + 16)
    big = torch.full((M, F + 9), 3.0, device="cuda")
    aux = torch.full((M, 2 * F + 3), 3.0, dtype=BF, device="cuda")
    ck, exp = torch.full((M, 2 * F + 5), 9, dtype=U8, device="cuda"), torch.full((M, 2 * nb + 3), 9, dtype=U8, device="cuda")
    keep = dict(aux=aux[:, 1:1 + 2 * F]) if kept == "bf16" else dict(ck=ck[:, 3:3 + 2 * F], ck_exp=exp[:, 1:1 + 2 * nb])
    ws = torch.empty(L.fp8_gated_linear_workspace(M, F, K, 5, 5), dtype=U8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    L.fp8_gated_linear(A, 0, 5, sa, B, 0, 5, sb, big[:, 4:4 + F], act=4, workspace=ws, stream=s, **keep)
    s.synchronize()
    (x, Ex), (o, Eo) = G.forward(*R.product(A, 0, 5, sa, B, 0, 5, sb), None, 4)
    R.close(big[:, 4:4 + F], o, Eo)
    assert bool((big[:, :4] == 3).all()) and bool((big[:, 4 + F:] == 3).all())
    if kept == "bf16":
        R.close(aux[:, 1:1 + 2 * F], x, Ex)
        assert bool((aux[:, 0] == 3).all()) and bool((aux[:, 1 + 2 * F:] == 3).all())
        x = aux[:, 1:1 + 2 * F]
    else:
        for h in (0, 1):
            c, e = ck[:, 3 + h * F:3 + h * F + F], exp[:, 1 + h * nb:1 + h * nb + nb]
            G.close_checkpoint(c, e, x[:, h * F:h * F + F], Ex[:, h * F:h * F + F])
        for t, a, n in ((ck, 3, 2 * F), (exp, 1, 2 * nb)):
            assert bool((t[:, :a] == 9).all()) and bool((t[:, a + n:] == 9).all())
        x = torch.cat([G.load(ck[:, 3:3 + F], exp[:, 1:1 + nb]), G.load(ck[:, 3 + F:3 + 2 * F], exp[:, 1 + nb:1 + 2 * nb])], 1)
    A, sa = operand(g, M, K, 1, 5, 1.0, K + 16)
    B, sb = operand(g, F, K, 0, 0, 0.08, K + 48)
    big8 = torch.full((M, 2 * F + 8), 9, dtype=U8, device="cuda")
    scale = torch.full((1,), 50.0, device="cuda")
    ws = torch.empty(L.fp8_gated_linear_workspace(M, F, K, 5, 0, True), dtype=U8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with pytest.raises(L.Fp8Error) as refused:      # D starts on a dword, as fp8_scaled_gemm's
        L.fp8_gated_linear(A, 1, 5, sa, B, 0, 0, sb, big8[:, 3:3 + 2 * F], act=4, backward=True, d_fmt=0, d_scale=scale, workspace=ws, stream=s,
                           **keep)
    assert refused.value.status == 3
    codes = big8[:, 4:4 + 2 * F]
    L.fp8_gated_linear(A, 1, 5, sa, B, 0, 0, sb, codes, act=4, backward=True, d_fmt=0, d_scale=scale, workspace=ws, stream=s, **keep)
    s.synchronize()
    o, Eo = G.backward(*R.product(A, 1, 5, sa, B, 0, 0, sb), x, 4)
    R.close8(codes.contiguous(), 0, 50 * o, 50 * Eo)
    assert bool((big8[:, :4] == 9).all()) and bool((big8[:, 4 + 2 * F:] == 9).all())
    with pytest.raises(ValueError):                 # a workspace of its own, on a stream of its own
        L.fp8_gated_linear(A, 1, 5, sa, B, 0, 0, sb, codes, act=4, backward=True, d_fmt=0, d_scale=scale, stream=s, **keep)


@pytest.mark.parametrize("size", [(4, 640, 4096), (300, 520, 1024), (2048, 2048, 512)])
def test_repeatable_and_graph(L, size):
    """The pair forward and back out of one graph, a checkpoint between them."""
    M, F, K = size
    g, nb = gen(2), G.blocks(F)
    A, sa = operand(g, M, K, 0, 0)
    B, sb = operand(g, 2 * F, K, 0, 0, K ** -0.5)
    dA, dsa = operand(g, M, K, 1, 0)
    dB, dsb = operand(g, F, K, 0, 0, K ** -0.5)
    bias = rand(g, (2 * F,), 0.5)
    h, h_t = (torch.empty(s, dtype=U8, device="cuda") for s in ((M, F), (F, M)))
    d, d_t = (torch.empty(s, dtype=U8, device="cuda") for s in ((M, 2 * F), (2 * F, M)))
    ck, exp = torch.empty((M, 2 * F), dtype=U8, device="cuda"), torch.empty((M, 2 * nb), dtype=U8, device="cuda")
    db, amax, damax = torch.empty(2 * F, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    scale = torch.full((1,), 20.0, device="cuda")
    ws = torch.empty(max(16, *(L.fp8_gated_linear_workspace(M, F, K, 0, 0, b) for b in (False, True))), dtype=U8, device="cuda")

    def step():
        L.fp8_gated_linear(A, 0, 0, sa, B, 0, 0, sb, h, bias=bias, ck=ck, ck_exp=exp, d_fmt=0, d_scale=scale, D_t=h_t, d_amax=amax, workspace=ws)
        L.fp8_gated_linear(dA, 1, 0, dsa, dB, 0, 0, dsb, d, ck=ck, ck_exp=exp, backward=True, dbias=db, d_fmt=1, d_scale=scale, D_t=d_t,
                           d_amax=damax, workspace=ws)
        return [t.clone() for t in (h, h_t, ck, exp, d, d_t, db, amax, damax)]

    first = step()
    for a, b in zip(first, step()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(4):
        bias.normal_()
        ws.random_(0, 255)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i


# ---- every kernel, with values that are sums of few small integers (see
# test_gpu_gemm_epilogue_paths.py): products, their products with g and u (small
# powers of two) and column sums are exact, so that one lost row, part of K or bit shows

FEW, TILES, LARGE = 0, 1, 2
# rows, outputs, K, scalings, direction: kernel, rows of its tiles, whether K is cut
PATHS = [
    (3, 1000, 4112, (0, 0), False), (16, 520, 2064, (5, 5), False), (13, 264, 4096, (1, 2), False), (7, 330, 2048, (1, 2), False),
    (7, 328, 2048, (1, 1), False), (16, 136, 1024, (3, 4), False), (1, 8, 48, (0, 5), False),
    (33, 260, 656, (0, 0), False), (64, 256, 8192, (5, 0), False), (300, 260, 4112, (5, 5), False), (130, 136, 2048, (1, 2), False),
    (130, 128, 2048, (1, 2), False), (130, 132, 2048, (3, 4), False), (1037, 999, 2320, (5, 5), False), (1037, 1024, 2304, (1, 2), False),
    (1037, 1000, 2304, (1, 2), False), (1500, 1000, 384, (3, 4), False), (1500, 1000, 384, (2, 1), False), (300, 500, 4096, (1, 2), False),
    (300, 500, 4096, (3, 3), False), (2050, 2051, 656, (0, 0), False), (1100, 2052, 512, (5, 5), False), (2048, 2048, 512, (1, 2), False),
    (2048, 2048, 512, (2, 2), False), (2048, 2048, 512, (4, 3), False), (2048, 2048, 512, (0, 2), False),
    (2050, 4104, 640, (0, 0), False), (2050, 4104, 656, (0, 0), False), (2050, 4104, 640, (5, 5), False), (2050, 4104, 656, (0, 5), False),
    (2050, 4224, 640, (1, 2), False), (2050, 4104, 640, (1, 2), False), (2050, 4104, 640, (3, 4), False), (2050, 4224, 640, (3, 4), False),
    (3, 1000, 4112, (0, 0), True), (16, 520, 2064, (5, 5), True), (13, 264, 4096, (1, 2), True), (16, 136, 1024, (3, 4), True),
    (33, 520, 656, (0, 0), True), (64, 512, 8192, (5, 0), True), (300, 520, 4112, (5, 5), True), (130, 264, 2048, (1, 2), True),
    (130, 264, 2048, (1, 1), True), (1037, 1999, 2320, (5, 5), True), (1037, 1999, 2304, (1, 2), True), (1500, 2000, 384, (3, 4), True),
    (300, 1000, 4096, (3, 3), True), (2050, 4103, 656, (0, 0), True), (2048, 4096, 512, (2, 2), True), (2050, 4104, 640, (0, 0), True),
    (2050, 4104, 656, (5, 5), True), (2050, 4104, 640, (5, 0), True), (2050, 4104, 656, (0, 0), True), (2050, 4104, 640, (1, 2), True),
    (2050, 4104, 640, (3, 4), True)]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("out", ["f32", "bf16", "fp8"])
def test_exact_on_each_kernel(L, taken, path, out):
    M, F, K, (asc, bsc), back = path
    for kept in ("ckpt", "bf16"):
        g = torch.Generator(device="cuda").manual_seed(M + F + K + asc)
        n, nb = (2 * F if back else F), G.blocks(F)
        A, sa, a = small(g, M, K, int(back), asc)
        B, sb, b = small(g, F if back else 2 * F, K, 0, bsc)
        v = torch.matmul(a, b.t())
        D = Guarded((M, n), {"f32": F32, "bf16": BF, "fp8": U8}[out])
        amax, kw = Guarded((1,), F32), {"act": L.ACT_RELU, "backward": back}
        fmt, f8, top, scale = (1, torch.float8_e5m2, 57344.0, 4.0) if back else (0, torch.float8_e4m3fn, 448.0, 0.25)
        if out == "fp8":
            D_t = Guarded((n, M), U8)
            kw.update(d_fmt=fmt, d_scale=torch.full((1,), scale, device="cuda"), D_t=D_t.t)
        if back:
            x = torch.tensor([-2.0, -1.0, 1.0, 2.0], device="cuda")[torch.randint(0, 4, (M, 2 * F), generator=g, device="cuda")]
            db = Guarded((2 * F,), F32)
            kw["dbias"] = db.t
            if kept == "bf16":
                kw["aux"] = x.to(BF)
            else:
                parts = [G.save(x[:, :F]), G.save(x[:, F:])]
                kw["ck"], kw["ck_exp"] = (torch.cat(t, 1) for t in zip(*parts))
            gate, up = x[:, :F].double(), x[:, F:].double()
            want = torch.cat([v * up * (gate > 0), v * gate.clamp(min=0)], 1)
        else:
            bias = torch.randint(-8, 9, (2 * F,), generator=g, device="cuda").float()
            u = v + bias.double()
            kw["bias"] = bias
            if kept == "bf16":
                aux = Guarded((M, 2 * F), BF)
                kw["aux"] = aux.t
            else:
                ck, exp = Guarded((M, 2 * F), U8), Guarded((M, 2 * nb), U8)
                kw["ck"], kw["ck_exp"] = ck.t, exp.t
            # (one product of the two integers: binary32 rounds it once)
            want = (u[:, :F].clamp(min=0) * u[:, F:]).float().double()
        L.fp8_gated_linear(A, int(back), asc, sa, B, 0, bsc, sb, D.t, d_amax=amax.t, **kw)
        torch.cuda.synchronize()
        say("gated exact", path, out, kept, taken[-1])
        D.check(), amax.check()
        if out == "fp8":
            D_t.check()
            assert torch.equal(D.t.view(f8).float(), (want * scale).clamp(-top, top).float().to(f8).float())
            assert torch.equal(D_t.t, D.t.t())
        else:
            assert torch.equal(D.t, want.float().to(D.t.dtype))
        assert float(amax.t) == float((want.float().to(BF) if out == "bf16" else want.float()).abs().max())
        if back:
            db.check()
            assert torch.equal(db.t, want.sum(0).float())
        elif kept == "bf16":
            aux.check()
            assert torch.equal(aux.t, u.float().to(BF))
        else:
            ck.check(), exp.check()
            for h in (0, 1):
                q, e = G.save(u[:, h * F:(h + 1) * F].float())
                assert torch.equal(ck.t[:, h * F:(h + 1) * F], q) and torch.equal(exp.t[:, h * nb:(h + 1) * nb], e)


@pytest.mark.parametrize("p", [BF, F32])
@pytest.mark.parametrize("M,K", [(1, 128), (16, 4096), (17, 256), (32, 272), (20, 8192), (33, 256)])
def test_bias_gradient_of_few_rows(L, M, K, p):
    """dbias of up to 32 rows has no join; it may start on any element."""
    F = 203
    g = gen(M + K)
    A, sa = operand(g, M, K, 1, 0)
    B, sb = operand(g, F, K, 0, 0, 0.5 / K ** 0.5)
    aux = rand(g, (M, 2 * F), 1.5).to(BF)
    D = torch.empty((M, 2 * F), device="cuda")
    for first in (0, 1, 3):
        whole = torch.full((2 * F + 8,), 3.0, dtype=p, device="cuda")
        db = whole[first:first + 2 * F]
        say("gated dbias", M, K, p, first)
        L.fp8_gated_linear(A, 1, 0, sa, B, 0, 0, sb, D, aux=aux, backward=True, dbias=db)
        torch.cuda.synchronize()
        o, Eo = G.backward(*R.product(A, 1, 0, sa, B, 0, 0, sb), aux, 4)
        R.close(db, o.sum(0), Eo.sum(0) + (R.C + M * 2.0 ** -24) * o.abs().sum(0))
        assert bool((whole[:first] == 3).all()) and bool((whole[first + 2 * F:] == 3).all())
