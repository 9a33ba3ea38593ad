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
