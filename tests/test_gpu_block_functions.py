"""The functions inside the operators around the linears, one value at a time and
relative to that value, where their 64-bit forms say how large it is: the tails
of an activation, gates that are all but closed, turns next to a quarter.

Bounds count roundings of binary32 (u = 2^-24, half a step).  The hardware
exponential and reciprocal are within a step each (2 u)."""
import math

import pytest
import torch

from gpu_util import Guarded, say

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
u = 2.0 ** -24


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


def norm_cdf(t):
    return 0.5 * torch.special.erfc(-t * math.sqrt(0.5))


@pytest.mark.parametrize("rows", [1, 40])
def test_gelu_keeps_its_digits_in_the_tail(L, rows):
    """GELU and its slope from -13 to 13.  The exponential's argument u^2 / 2 is
    rounded three times (the constant, two products): 3 u^2 / 2 roundings of the
    result; 24 more for the exponential, the reciprocal, a fit within 2 u, its
    eight steps and the products around it."""
    x = torch.cat([torch.linspace(-13, 13, 4096, device="cuda"), torch.tensor([-1e-6, 0.0, 1e-20, 30.0, 1e6], device="cuda")]).to(BF).float()
    N = x.numel()
    empty = torch.empty((rows, 0), dtype=U8, device="cuda")
    D = Guarded((rows, N), F32)
    L.fp8_scaled_gemm_ep(empty, 0, 0, None, torch.empty((N, 0), dtype=U8, device="cuda"), 0, 0, None, D.t, bias=x, act=L.ACT_GELU)
    torch.cuda.synchronize()
    D.check()
    t = x.double()
    want = t * norm_cdf(t)
    assert bool(((D.t.double() - want).abs() <= (24 + 1.5 * t * t) * u * want.abs() + 2.0 ** -126).all())
    # the slope: a product of ones (1 * 1 + 0 + ...), times act'(x)
    A, B = torch.zeros((rows, 16), dtype=U8, device="cuda"), torch.zeros((N, 16), dtype=U8, device="cuda")
    A[:, 0], B[:, 0] = 0x38, 0x38
    one = torch.ones(1, device="cuda")
    aux = x.to(BF).expand(rows, N).contiguous()
    L.fp8_scaled_gemm_ep(A, 0, 0, one, B, 0, 0, one, D.t, act=L.ACT_GELU, aux=aux, backward=True)
    torch.cuda.synchronize()
    D.check()
    pdf = torch.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)
    room = (24 + 1.5 * t * t) * u * (norm_cdf(t) + t.abs() * pdf) + 2.0 ** -126
    assert bool(((D.t.double() - (norm_cdf(t) + t * pdf)).abs() <= room).all())


@pytest.mark.parametrize("inverse", [False, True])
def test_turns_keep_their_digits_next_to_a_quarter(L, inverse):
    """Heads (1, 0) turned far into a context: cosine and sine within 3 steps of
    themselves (two of the hardware's function, one of the correction), however
    close to 0."""
    T, n = 5000, 64
    freqs = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    q = torch.zeros((T, 1, 2 * n), device="cuda")
    q[..., :n] = 1
    L.fp8_rope(q, freqs, pos, inverse=inverse)
    torch.cuda.synchronize()
    # the turn's fraction, in 64 bits as the definition has it, then to a quarter: cos and sin of small angles
    a = pos.double()[:, None] * freqs
    c, s = a.cos(), a.sin() * (-1 if inverse else 1)
    # (position times frequency in 64 bits leaves 2^-52 of up to 2^20 radians)
    room = 2.0 ** -30
    assert bool(((q[:, 0, :n].double() - c).abs() <= 6 * u * c.abs() + room).all())
    assert bool(((q[:, 0, n:].double() - s).abs() <= 6 * u * s.abs() + room).all())


@pytest.mark.parametrize("act", [1, 2])
@pytest.mark.parametrize("gate", ["token", "channel"])
def test_gate_gradients_keep_their_digits(L, act, gate):
    """Gates from -12 to 12, through a sigmoid (1) or a tanh (2): the derivative
    is e / (1 + e)^2 (times 4), e = exp(-|g|) (exp(-2 |g|)), to 12 roundings and
    two of e's argument, beside the sums of 64 columns or rows."""
    rows, cols = (513, 64) if gate == "token" else (64, 513)
    g = torch.Generator(device="cuda").manual_seed(act)
    z = torch.randn((rows, cols), generator=g, device="cuda").abs().add(0.5).to(BF)   # one sign: nothing cancels
    dh = torch.rand((rows, cols), generator=g, device="cuda") + 0.5
    x = torch.linspace(-12, 12, 513, device="cuda")
    gate_t = x.view(rows, 1).contiguous() if gate == "token" else x
    dg, dx = torch.empty_like(gate_t), torch.empty_like(dh)
    rz = torch.rsqrt(z.double().square().mean(1, keepdim=True) + 1e-6)
    stats = torch.cat([torch.zeros_like(rz), rz], 1).float()
    L.fp8_block_norm_bwd(dh, dx, dh=dh, z=z, gate=gate_t, gate_act=act, stats_z=stats, dgate=dg)
    torch.cuda.synchronize()
    t = gate_t.double()
    e = torch.exp(-t.abs() * (1 if act == 1 else 2))
    slope = (1 if act == 1 else 4) * e / (1 + e) ** 2
    n = z.double() * stats[:, 1:].double()
    want = slope * (dh.double() * n).sum(1 if gate == "token" else 0, keepdim=gate == "token")
    say(float(((dg.double() - want).abs() / want).max()))
    assert bool(((dg.double() - want).abs() <= (12 + 64 + 4 * t.abs()) * u * want).all())


def test_broadcast_heads_are_read_but_not_written(L):
    """A key head that several query heads share, as an expanded view: turned
    into its own memory it is right, in place it would be turned once per head."""
    x = torch.randn((20, 1, 16), device="cuda")
    freqs = torch.linspace(1.0, 0.1, 8, dtype=torch.float64, device="cuda")
    q, wide = torch.randn((20, 4, 16), device="cuda"), x.expand(20, 4, 16)
    qo, ko, one = torch.empty_like(q), torch.empty_like(q), torch.empty_like(x)
    L.fp8_rope(q, freqs, k=wide, q_out=qo, k_out=ko)
    L.fp8_rope(x, freqs, q_out=one)
    assert torch.equal(ko, one.expand(20, 4, 16))
    before = x.clone()
    for kw in (dict(k=wide, q_out=qo), dict(k=q, q_out=wide, k_out=ko)):
        with pytest.raises(ValueError, match="broadcast"):
            L.fp8_rope(q, freqs, **kw)
    with pytest.raises(ValueError, match="broadcast"):
        L.fp8_rope(x[:1].expand(20, 1, 16), freqs)
    assert torch.equal(x, before)
