"""The example's block with a gated feed-forward part, its activations kept in 8 bits: a
training step against 64-bit autograd of the unquantised block, and tokens decoded one by
one.

Tolerances count roundings to 8 bits as test_gpu_transformer_block.py does.  What the
feed-forward part's first product gets, it passes on through both factors: with g and w of
unit variance, h = silu(g) w changes by silu'(g) w dg + silu(g) dw, in the mean square
(0.38 + 0.36) / 0.36 = 2.1 times the relative error, so y1 and w1 count twice, and so do
the roundings of the kept g and w in the gradients."""
import pytest
import torch

from test_gpu_transformer_block import attention64, example, near

pytestmark = pytest.mark.gpu


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
    g, w = (norm(h, p["n1"]) @ p["w1"].t() + p["b1"]).chunk(2, 1)
    return h + (torch.nn.functional.silu(g) * w) @ p["w2"].t()


# y0, o, u, wqkv, wo, w2, and y1, w1 twice
OUT = 10
# the same again; g | w (twice) and the branch, kept in 8 bits
GRAD = 2 * OUT + 3


@pytest.mark.parametrize("tokens,hidden,heads,kv,dim,ffn", [(64, 256, 4, 2, 64, 512), (208, 384, 6, 6, 64, 1104),
                                                            (16, 320, 5, 1, 64, 880)])
def test_training_step(tokens, hidden, heads, kv, dim, ffn):
    b = example().Block(hidden, heads, kv, dim, ffn, gated=True)
    g = torch.Generator(device="cpu").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    dout = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    for _ in range(3):   # delayed scaling: the amax values of the first steps set the scales
        out, s = b.forward(x.cuda())
        assert "aux" not in s and "a" not in s
        dx, grads = b.backward(dout.cuda(), s)
        b.step()
    p = {n: t.double().cpu().requires_grad_() for n, t in b.param.items()}
    x64 = x.double().requires_grad_()
    want = plain(b, p, x64)
    want.backward(dout.double())
    near(out, want.detach(), OUT, 0, "out")
    near(dx, x64.grad, GRAD, 4, "dx")
    for n in grads:
        near(grads[n], p[n].grad, GRAD, 4, n)


def test_decode_one_by_one():
    m = example()
    tokens, hidden, heads, kv, dim, ffn = 12, 256, 4, 2, 64, 512
    b = m.Block(hidden, heads, kv, dim, ffn, gated=True)
    x = torch.randn(tokens, hidden, generator=torch.Generator(device="cpu").manual_seed(2)).to(torch.bfloat16)
    caches = [torch.zeros(tokens, kv, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    one = torch.cat([b.decode(x[i:i + 1].cuda(), i, *caches) for i in range(tokens)])
    p = {n: t.double().cpu() for n, t in b.param.items()}
    near(one, plain(b, p, x.double()), OUT, 0, "out")
    rest = b.decode(x[5:].cuda(), 5, *[c.clone() for c in caches])
    near(rest, plain(b, p, x.double())[5:], OUT, 0, "out")
