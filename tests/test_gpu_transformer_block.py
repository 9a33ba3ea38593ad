"""The example's block as a whole: a training step against 64-bit autograd of
the unquantised block, and tokens decoded one by one against the same block.

Tolerances are on ||got - want|| / ||want||.  A rounding to E4M3 moves a value
by at most 2^-4 of it, evenly spread over +-half a step: at most 2^-4 / sqrt(3)
in the mean square (E5M2: 2^-3 / sqrt(3)); roundings of different values are
independent, so the squares of successive layers add.  A layer that keeps the
norm of what passes (products with weights of unit gain, norms, rotations) adds
its roundings once; the feed-forward's and the gate's slopes and the softmax
pass less than twice what they get, so every count below is taken twice."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "transformer_block.py")
E4, E5 = (2.0 ** -4) ** 2 / 3, (2.0 ** -3) ** 2 / 3


def example():
    spec = importlib.util.spec_from_file_location("transformer_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def attention64(q, k, v):
    q, k, v = (t.transpose(0, 1) for t in (q, k, v))
    rep = q.shape[0] // k.shape[0]
    k, v = k.repeat_interleave(rep, 0), v.repeat_interleave(rep, 0)
    s = torch.matmul(q, k.transpose(1, 2).contiguous()) * q.shape[2] ** -0.5
    s = s.masked_fill(torch.ones_like(s[0], dtype=torch.bool).triu(1), float("-inf"))
    return torch.matmul(s.softmax(-1), v).transpose(0, 1)


def plain(b, p, x):
    """The block in 64 bits, on the CPU, from the unquantised weights."""
    def norm(t, w):
        return t * torch.rsqrt((t * t).mean(1, keepdim=True) + 1e-6) * w

    def turn(t):
        a = torch.arange(t.shape[0], dtype=torch.float64)[:, None, None] * b.freqs.cpu()
        c, s = a.cos(), a.sin()
        u, w = t.chunk(2, -1)
        return torch.cat((u * c - w * s, w * c + u * s), -1)

    n = x.shape[0]
    qkv = (norm(x, p["n0"]) @ p["wqkv"].t()).view(n, -1, b.dim)
    q, k, v = qkv.split((b.heads, b.kv, b.kv), 1)
    a = attention64(turn(q), turn(k), v).reshape(n, -1) @ p["wo"].t()
    h = x + torch.tanh(p["gate"]) * norm(a, p["na"])
    u = torch.nn.functional.gelu(norm(h, p["n1"]) @ p["w1"].t() + p["b1"])
    return h + u @ p["w2"].t()


def near(got, want, e4, e5, name):
    got = got.detach().double().cpu()
    err = float((got - want).norm() / want.norm())
    lim = (2 * (e4 * E4 + e5 * E5)) ** 0.5
    assert err <= lim, f"{name}: off by {err:.3f}, at most {lim:.3f}"


@pytest.mark.parametrize("tokens,hidden,heads,kv,dim,ffn", [(64, 256, 4, 2, 64, 512), (208, 384, 6, 6, 64, 1104)])
def test_training_step(tokens, hidden, heads, kv, dim, ffn):
    b = example().Block(hidden, heads, kv, dim, ffn)
    g = torch.Generator(device="cpu").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    dout = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    for _ in range(3):   # delayed scaling: the amax values of the first steps set the scales
        out, s = b.forward(x.cuda())
        dx, grads = b.backward(dout.cuda(), s)
        b.step()
    p = {n: t.double().cpu().requires_grad_() for n, t in b.param.items()}
    x64 = x.double().requires_grad_()
    want = plain(b, p, x64)
    want.backward(dout.double())
    # y0, o, y1, u and the four weights; a gradient: the same again, and its own
    near(out, want.detach(), 8, 0, "out")
    near(dx, x64.grad, 16, 4, "dx")
    for n in grads:
        near(grads[n], p[n].grad, 16, 4, n)


def test_decode_one_by_one():
    m = example()
    tokens, hidden, heads, kv, dim, ffn = 12, 256, 4, 2, 64, 512
    b = m.Block(hidden, heads, kv, dim, ffn)
    x = torch.randn(tokens, hidden, generator=torch.Generator(device="cpu").manual_seed(2)).to(torch.bfloat16)
    caches = [torch.zeros(tokens, kv, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    one = torch.cat([b.decode(x[i:i + 1].cuda(), i, *caches) for i in range(tokens)])
    p = {n: t.double().cpu() for n, t in b.param.items()}
    near(one, plain(b, p, x.double()), 8, 0, "out")
    # several tokens at once, after others
    rest = b.decode(x[5:].cuda(), 5, *[c.clone() for c in caches])
    near(rest, plain(b, p, x.double())[5:], 8, 0, "out")
