"""How far a checkpoint's values may be off, at maxima of every exponent of binary32: half a step of
the code, which is 2^-4 of a value, or 2^-17 of its block's largest, or, where the block's power of two
is at its end, half of E4M3's smallest step times 2^-126."""
import pytest
import torch

import gated_ref as G
from gpu_util import say

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


@pytest.mark.parametrize("dtype", [BF, F32])
def test_accuracy_at_every_exponent(L, dtype):
    say("checkpoint accuracy", dtype)
    e = torch.arange(-149 if dtype == F32 else -133, 128, device="cuda", dtype=torch.float64)
    top = torch.cat([m * torch.exp2(e) for m in (1.0, 1.5, 1.75, 1.9921875)]).to(dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (2 * torch.rand((top.numel(), 64), generator=g, device="cuda", dtype=torch.float64) - 1) * top.double()[:, None]
    x[:, 32:] *= 2.0 ** -20                            # a block far below its neighbour
    x = x.to(dtype)
    x[:, 7] = top
    ck, exp = torch.empty(x.shape, dtype=U8, device="cuda"), torch.empty((x.shape[0], 2), dtype=U8, device="cuda")
    y = torch.empty(x.shape, device="cuda")
    L.fp8_checkpoint_save(x, ck, exp)
    L.fp8_checkpoint_load(ck, exp, y)
    torch.cuda.synchronize()
    v, want = x.double(), G.load(ck, exp)
    far = v.abs() >= 1.9375 * 2.0 ** 127               # (their codes stand for 2^128)
    assert bool((want[far].abs() == 2.0 ** 128).all()) and bool((y[far].abs() == float("inf")).all()) and int(far.sum()) > 0
    assert torch.equal(y[~far].double(), want[~far])   # exact in binary32
    y = want
    largest = G.spread(G.block_max(v), 64)
    lim = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -17 * largest).clamp(min=2.0 ** -136)
    bad = (y - v).abs() > lim
    assert not bool(bad.any()), f"{int(bad.sum())} values off, the first at {bad.nonzero()[0].tolist()}"
    # the last term is needed where the block's largest value is below 2^-118, and nowhere else; not for BF16,
    # whose smallest step, 2^-133, is four of the code's times 2^-126
    tight = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -17 * largest)
    beyond = (y - v).abs() > tight
    assert bool(beyond.any()) == (dtype == F32) and bool((largest[beyond] < 2.0 ** -118).all())
