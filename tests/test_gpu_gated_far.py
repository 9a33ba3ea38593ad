"""The gated pair and checkpoints where offsets pass 2^32: sums of few small integers, exact, on rows at
the start, around the 2^31st and the 2^32nd byte and at the end; bias gradients over all rows."""
import pytest
import torch

import gated_ref as G
from gpu_util import say
from test_gpu_gated import LARGE, L, taken      # noqa: F401  (fixtures)
from test_gpu_gemm_epilogue_paths import small

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
M, K = 81920, 128
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def parts(cols, rows=M):
    """Slices of rows of `cols` bytes."""
    at = sorted({0, rows - 128} | {min(rows - 128, max(0, (1 << b) // cols - 64)) for b in (31, 32)})
    return [slice(a, a + 128) for a in at]


def codes(want, scale, f8, top):
    return (want * scale).clamp(-top, top).float().to(f8).float()


@pytest.mark.parametrize("F,kernel", [(28672, (LARGE, 256, False)), (28671, None)])
def test_forward(L, taken, F, kernel):
    nb = G.blocks(F)
    g = torch.Generator(device="cuda").manual_seed(F)
    A, sa, a = small(g, M, K, 0, 0)
    B, sb, b = small(g, 2 * F, K, 0, 0)
    D, D_t = torch.empty((M, F), dtype=U8, device="cuda"), torch.empty((F, M), dtype=U8, device="cuda")
    ck, exp = torch.empty((M, 2 * F), dtype=U8, device="cuda"), torch.empty((M, 2 * nb), dtype=U8, device="cuda")
    aux = torch.empty((M, 2 * F), dtype=BF, device="cuda")
    say("gated far forward", F)
    L.fp8_gated_linear(A, 0, 0, sa, B, 0, 0, sb, D, act=L.ACT_RELU, aux=aux, ck=ck, ck_exp=exp, d_fmt=0,
                       d_scale=torch.full((1,), 0.25, device="cuda"), D_t=D_t)
    torch.cuda.synchronize()
    assert kernel is None or taken == [kernel]
    for r in parts(2 * F):
        v = torch.matmul(a[r], b.t())
        want = codes((v[:, :F].clamp(min=0) * v[:, F:]).float().double(), 0.25, E4, 448)
        assert torch.equal(D[r].view(E4).float(), want) and torch.equal(D_t[:, r].t(), D[r])
        assert torch.equal(aux[r], v.float().to(BF))
        for h in (0, 1):
            q, e = G.save(v[:, h * F:(h + 1) * F].float())
            assert torch.equal(ck[r, h * F:(h + 1) * F], q) and torch.equal(exp[r, h * nb:(h + 1) * nb], e)


@pytest.mark.parametrize("F,kernel", [(28672, (LARGE, 256, False)), (28671, None)])
@pytest.mark.parametrize("kept", ["ckpt", "bf16"])
def test_backward(L, taken, F, kernel, kept):
    nb = G.blocks(F)
    g = torch.Generator(device="cuda").manual_seed(F + 1)
    A, sa, a = small(g, M, K, 1, 0)
    B, sb, b = small(g, F, K, 0, 0)
    ck = torch.tensor([0x70, 0x78, 0xF0, 0xF8], dtype=U8, device="cuda")[torch.randint(0, 4, (M, 2 * F), generator=g, device="cuda",
                                                                                      dtype=torch.int32)]   # 128, 256, negative
    exp = torch.full((M, 2 * nb), 120, dtype=U8, device="cuda")                                             # 2^-7
    kw = dict(ck=ck, ck_exp=exp) if kept == "ckpt" else dict(aux=(ck.view(E4).to(BF) / 128))
    D, D_t = torch.empty((M, 2 * F), dtype=U8, device="cuda"), torch.empty((2 * F, M), dtype=U8, device="cuda")
    db, amax = torch.empty(2 * F, device="cuda"), torch.empty(1, device="cuda")
    say("gated far backward", F, kept)
    L.fp8_gated_linear(A, 1, 0, sa, B, 0, 0, sb, D, act=L.ACT_RELU, backward=True, dbias=db, d_fmt=1, d_scale=torch.full((1,), 4.0, device="cuda"),
                       D_t=D_t, d_amax=amax, **kw)
    torch.cuda.synchronize()
    assert kernel is None or taken == [kernel]

    def formula(r):
        v, x = torch.matmul(a[r], b.t()), ck[r].view(E4).double() / 128
        gate, up = x[:, :F], x[:, F:]
        return torch.cat([v * up * (gate > 0), v * gate.clamp(min=0)], 1)
    for r in parts(2 * F):
        assert torch.equal(D[r].view(E5).float(), codes(formula(r), 4.0, E5, 57344)) and torch.equal(D_t[:, r].t(), D[r])
    total, size, top = 0.0, 0.0, 0.0
    for m in range(0, M, 4096):
        w = formula(slice(m, m + 4096))
        total, size, top = total + w.sum(0), size + w.abs().sum(0), max(top, float(w.abs().max()))
    assert float(size.max()) < 2 ** 24, "column sums are exact"
    assert torch.equal(db, total.float()) and float(amax) == top


@pytest.mark.parametrize("dtype", [BF, F32])
def test_checkpoint(L, dtype):
    rows, cols = 70001, 65538
    nb = G.blocks(cols)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((rows, cols), dtype=dtype, device="cuda").normal_(generator=g)
    ck, exp = torch.empty((rows, cols), dtype=U8, device="cuda"), torch.empty((rows, nb), dtype=U8, device="cuda")
    y = torch.empty_like(x)
    say("checkpoint far", dtype)
    L.fp8_checkpoint_save(x, ck, exp)
    L.fp8_checkpoint_load(ck, exp, y)
    torch.cuda.synchronize()
    for r in parts(cols, rows) + parts(cols * x.element_size(), rows):
        q, e = G.save(x[r])
        assert torch.equal(ck[r], q) and torch.equal(exp[r], e)
        assert torch.equal(y[r].double(), G.load(q, e))
