"""fp8_rope and fp8_rope_freqs against their 64-bit forms (block_ref.py)."""
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


def check(got, x, pos, freqs, inter, inv, scale):
    want, S = R.rope(x, pos, freqs, inter, inv, scale)
    n = 2 * freqs.numel()
    # cosine and sine of a turn rounded to binary32 (2 pi 2^-25) within 2
    # units, scaled; two products and a sum
    R.close(got[..., :n], want[..., :n], 12 * 2.0 ** -24 * S[..., :n])
    assert torch.equal(got[..., n:], x[..., n:])


CASES = [(1, 1, 1, 2, 1), (1, 64, 8, 128, 64), (3, 5, 2, 80, 13), (7, 8, 8, 64, 32), (65, 3, 1, 96, 24), (130, 16, 4, 256, 128),
         (16, 64, 8, 128, 64), (1001, 7, 2, 63, 31), (20, 2, 1, 512, 200), (2, 300, 1, 64, 32), (5, 2, 0, 40, 0), (2, 1, 1, 2048, 1024)]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope(L, case, inter, dtype):
    T, H, KV, dim, n = case
    say("rope", case, inter, dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(T + dim)
    qkv = torch.randn((T, H + 2 * KV, dim), generator=g, device="cuda").to(dtype)
    q, k = qkv[:, :H], qkv[:, H:H + KV]
    freqs = R.rope_freqs(n, 10000.0, 0, 1, 1, 1, 2).cuda()
    inv, scale = T % 2, 1.0 if T % 3 else 1.25
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=[torch.int32, torch.int64][dim % 2])
    qo, ko = Guarded((T, H, dim), dtype), Guarded((T, KV, dim), dtype)
    kw = dict(positions=pos, layout=inter, inverse=bool(inv), scale=scale)
    L.fp8_rope(q, freqs, k=k if KV else None, q_out=qo.t, k_out=ko.t if KV else None, **kw)
    torch.cuda.synchronize()
    qo.check(), ko.check()
    check(qo.t, q, pos, freqs, inter, inv, scale)
    if KV:
        check(ko.t, k, pos, freqs, inter, inv, scale)
    before = qkv.clone()
    L.fp8_rope(q, freqs, k=k if KV else None, **kw)   # in place, inside the QKV tensor
    assert torch.equal(q, qo.t) and (KV == 0 or torch.equal(k, ko.t))
    assert torch.equal(qkv[:, H + KV:], before[:, H + KV:])


def test_default_positions_offset_and_far(L):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((9, 2, 32), generator=g, device="cuda")
    freqs = R.rope_freqs(16, 500000.0, 0, 1, 1, 1, 2).cuda()
    y = torch.empty_like(x)
    L.fp8_rope(x, freqs, q_out=y, offset=3)
    check(y, x, torch.arange(9, device="cuda") + 3, freqs, 0, 0, 1.0)
    L.fp8_rope(x, freqs, q_out=y, offset=(1 << 33))   # past 32 bits
    check(y, x, torch.arange(9, device="cuda") + (1 << 33), freqs, 0, 0, 1.0)
    L.fp8_rope(x, freqs, torch.arange(9, device="cuda") - 4, q_out=y)
    check(y, x, torch.arange(9, device="cuda") - 4, freqs, 0, 0, 1.0)


@pytest.mark.parametrize("inter", [0, 1])
def test_inverse_is_the_gradient(L, inter):
    """<rope(x), y> = <x, rope^-1(y)> for float32 heads: the inverse call is the
    transpose, and, the turn being linear, a difference along y is exact."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x, y = (torch.randn((50, 4, 64), generator=g, device="cuda") for _ in range(2))
    freqs = R.rope_freqs(24, 10000.0, 0, 1, 1, 1, 2).cuda()
    a, b = torch.empty_like(x), torch.empty_like(x)
    L.fp8_rope(x, freqs, q_out=a, layout=inter, scale=1.2)
    L.fp8_rope(y, freqs, q_out=b, layout=inter, scale=1.2, inverse=True)
    lhs, rhs = (a.double() * y.double()).sum(), (x.double() * b.double()).sum()
    room = 16 * 2.0 ** -24 * 4 * 1.2 * float((x.double().abs() * y.double().abs()).norm())
    assert abs(float(lhs - rhs)) <= room


def test_empty_and_stream(L):
    f = torch.ones(4, dtype=torch.float64, device="cuda")
    L.fp8_rope(torch.empty((0, 3, 8), device="cuda"), f)
    x = torch.randn((300, 6, 8), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(x)
    L.fp8_rope(x, f, q_out=y, stream=s)
    s.synchronize()
    check(y, x, torch.arange(300, device="cuda"), f, 0, 0, 1.0)


@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
@pytest.mark.parametrize("pairs", [1, 2, 20, 64])
def test_freqs(L, scaling, pairs):
    f = torch.empty(pairs, dtype=torch.float64, device="cuda")
    L.fp8_rope_freqs(f, 500000.0, scaling, 8.0, 8192.0, 1.0, 4.0)
    want = R.rope_freqs(pairs, 500000.0, scaling, 8.0, 8192.0, 1.0, 4.0)
    assert bool(((f.cpu() - want).abs() <= 1e-13 * want).all())
