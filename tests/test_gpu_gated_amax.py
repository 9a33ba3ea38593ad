"""The amax of fp8_gated_linear's FP8 output, on each forward kernel: planted where the matrix
unit loses bits.  Of 448 and seven times 2^-6 in a group of eight products it keeps 448 alone,
2.4e-4 of the sum; here the sums are exact in binary32 (multiples of 2^-6 below 2^18), so the
amax is their product, rounded once, and the activation's rounding."""
import pytest
import torch

import block_ref as R
from gpu_util import Guarded, say
from test_gpu_gated import FEW, LARGE, TILES, L, taken      # noqa: F401  (fixtures)
from test_gpu_gemm_epilogue_paths import small

pytestmark = pytest.mark.gpu
U8 = torch.uint8

# rows, outputs, K, scalings, kernel, rows of its tiles (None: whichever), whether K is cut
PATHS = [
    (1, 1000, 1024, (5, 5), FEW, 16, False), (3, 33, 1024, (0, 0), FEW, 16, False), (16, 136, 1024, (1, 2), FEW, 16, False),
    (7, 330, 1024, (1, 1), FEW, 16, False), (33, 260, 256, (0, 0), TILES, None, False), (300, 520, 256, (5, 5), TILES, None, False),
    (130, 132, 1024, (3, 4), TILES, None, None), (64, 256, 8192, (5, 0), TILES, None, True), (130, 136, 2048, (1, 2), TILES, None, True),
    (1037, 999, 1024, (5, 5), TILES, None, None), (1037, 1000, 1024, (2, 1), TILES, None, None), (2050, 2051, 640, (0, 0), TILES, None, False),
    (316, 16032, 1024, (5, 0), LARGE, 160, False), (2052, 3552, 1040, (0, 0), LARGE, 256, False), (2052, 3584, 1024, (3, 4), LARGE, 256, False),
    (2052, 3584, 1024, (1, 2), LARGE, 256, False)]


def planted(M, F, K, scalings, at, seed):
    asc, bsc = scalings
    g = torch.Generator(device="cuda").manual_seed(seed)
    (A, sa, _), (B, sb, _) = small(g, M, K, 0, asc), small(g, 2 * F, K, 0, bsc)
    m, f = at
    A[m] = 0x08                      # 2^-6
    A[m, ::8] = 0x7E                 # 448
    B[f], B[F + f] = 0x38, 0x38      # 1
    return A, sa, B, sb


@pytest.mark.parametrize("path", PATHS)
def test_amax_is_exact(L, taken, path):
    M, F, K, (asc, bsc), kernel, rows, cut = path
    for i, at in enumerate([(0, 0), (M - 1, F - 1), (M // 2, F // 3), (M * 5 // 7, F * 6 // 7)]):
        A, sa, B, sb = planted(M, F, K, (asc, bsc), at, M + F + i)
        bias = torch.randint(-8, 9, (2 * F,), device="cuda").float() if i % 2 else None
        D, amax = Guarded((M, F), U8), Guarded((1,), torch.float32)
        amax.t.fill_(1e30)
        say("gated amax", path, at)
        L.fp8_gated_linear(A, 0, asc, sa, B, 0, bsc, sb, D.t, act=L.ACT_RELU, bias=bias, d_fmt=L.E4M3,
                           d_scale=torch.full((1,), 2.0 ** -24, device="cuda"), d_amax=amax.t)
        torch.cuda.synchronize()
        D.check(), amax.check()
        v = R.product(A, 0, asc, sa, B, 0, bsc, sb)[0]
        v = v if bias is None else v + bias.double()
        want = float((v[:, :F].clamp(min=0) * v[:, F:]).abs().max())
        assert want == float((v[at[0], at[1]] * v[at[0], F + at[1]]).abs()), "the planted one is the largest"
        # (its sums: K / 32 + 8 roundings, of which only those past 24 bits round at all)
        assert abs(float(amax.t) - want) <= ((2 * (K // 32 + 8) if K > 1024 else 4) * 2.0 ** -24) * want, at
        # beside what is there already
        for before in (want * 4, want / 4):
            amax.t.fill_(before)
            L.fp8_gated_linear(A, 0, asc, sa, B, 0, bsc, sb, D.t, act=L.ACT_RELU, bias=bias, d_fmt=L.E4M3,
                               d_scale=torch.full((1,), 2.0 ** -24, device="cuda"), d_amax=amax.t, amax_accumulate=True)
            assert abs(float(amax.t) - max(before, want)) <= ((2 * (K // 32 + 8) if K > 1024 else 4) * 2.0 ** -24) * max(before, want)
    for t in taken:
        assert t[0] == kernel and (rows is None or t[1] == rows) and (cut is None or t[2] == cut), t


@pytest.mark.parametrize("M,F,K", [(3, 40, 128), (40, 72, 128), (2052, 3552, 128), (316, 16032, 128)])
def test_amax_of_zeros_infinities_and_nan(L, M, F, K):
    one, scale = torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
    A, B = torch.zeros((M, K), dtype=U8, device="cuda"), torch.zeros((2 * F, K), dtype=U8, device="cuda")
    D, amax = torch.empty((M, F), dtype=U8, device="cuda"), torch.full((1,), 7.0, device="cuda")
    bias = torch.zeros(2 * F, device="cuda")

    def call():
        L.fp8_gated_linear(A, 0, 0, one, B, 0, 0, one, D, act=L.ACT_NONE, bias=bias, d_fmt=L.E4M3, d_scale=scale, d_amax=amax)
        return float(amax)
    assert call() == 0
    bias[F - 1], bias[2 * F - 1] = 3.0, -5.0
    assert call() == 15
    bias[1], bias[F + 1] = 1.0, float("-inf")
    assert call() == float("inf")
    bias[F // 2] = float("nan")
    assert call() != call()


def test_amax_without_rows_or_k(L):
    one, scale = torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
    for M, K, want in ((0, 128, 0.0), (5, 0, 6.0), (40, 0, 6.0)):
        F = 24
        bias = torch.zeros(2 * F, device="cuda")
        bias[F - 1], bias[2 * F - 1] = 2.0, -3.0
        amax = torch.full((1,), 7.0, device="cuda")
        L.fp8_gated_linear(torch.zeros((M, K), dtype=U8, device="cuda"), 0, 0, one if K else None,
                           torch.zeros((2 * F, K), dtype=U8, device="cuda"), 0, 0, one if K else None,
                           torch.empty((M, F), dtype=U8, device="cuda"), act=L.ACT_NONE, bias=bias, d_fmt=L.E4M3, d_scale=scale, d_amax=amax)
        assert float(amax) == want


def test_two_streams_add_to_one_amax(L):
    """Two calls at once, each with a workspace of its own, and the larger of their amaxes."""
    M, F, K = 300, 520, 1024
    streams = [torch.cuda.Stream() for _ in range(2)]
    scale = torch.full((1,), 2.0 ** -24, device="cuda")
    amax, each = torch.zeros(1, device="cuda"), torch.zeros(2, device="cuda")
    ops = [planted(M, F, K, (0, 0), (7, 11), s) for s in (1, 2)]
    ws = [torch.empty(L.fp8_gated_linear_workspace(M, F, K, 0, 0), dtype=U8, device="cuda") for _ in range(2)]
    D = [torch.empty((M, F), dtype=U8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (A, sa, B, sb), w, d, s in zip(ops, ws, D, streams):
            L.fp8_gated_linear(A, 0, 0, sa, B, 0, 0, sb, d, d_fmt=L.E4M3, d_scale=scale, d_amax=amax, amax_accumulate=True,
                               workspace=w, stream=s)
    for i, ((A, sa, B, sb), w, d, s) in enumerate(zip(ops, ws, D, streams)):
        L.fp8_gated_linear(A, 0, 0, sa, B, 0, 0, sb, d, d_fmt=L.E4M3, d_scale=scale, d_amax=each[i:i + 1], workspace=w, stream=s)
    torch.cuda.synchronize()
    assert float(amax) == float(each.max()) > 0
