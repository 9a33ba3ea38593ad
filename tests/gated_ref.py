"""Plain 64-bit forms of the gated feed-forward pair and of 8-bit checkpoints, and
the error bounds that their kernels are held to (counted as in block_ref.py)."""
import torch

import block_ref as R

BLOCK = 32


def blocks(cols):
    return -(-cols // BLOCK)


def block_max(x):
    """max |x| of each block [rows][blocks]; NaN where one is in it."""
    return torch.stack([b.abs().amax(1) for b in torch.split(x, BLOCK, 1)], 1)


def spread(per_block, cols):
    return per_block.repeat_interleave(BLOCK, 1)[:, :cols]


def exponent(a):
    """e of a block from its largest magnitude, by trial: the largest |e| <= 126 with a 2^e <= 448."""
    a = a.double()
    e = torch.full(a.shape, -126, dtype=torch.int64, device=a.device)
    for k in range(-125, 127):
        e = torch.where(a * 2.0 ** k <= 448, k, e)
    return torch.where(a.isfinite() & (a > 0), e, 0)


def save(x):
    """(codes, bytes) of a checkpoint of x, exactly."""
    e = exponent(block_max(x.double()))
    v = x.double() * torch.exp2(spread(e, x.shape[1]).double())     # exact: a power of two, far from binary64's ends
    q = torch.where(v.isnan(), v, v.clamp(-448, 448)).float().to(R.F8[0]).view(torch.uint8)
    q = torch.where(v.isnan(), 0x7F | (128 * torch.signbit(x)).to(torch.uint8), q)
    return q, (127 - e).to(torch.uint8)


def load(ck, exp):
    """The values of a checkpoint in 64 bits."""
    w = torch.where(exp == 255, float("nan"), torch.exp2(exp.double() - 127))
    return ck.contiguous().view(R.F8[0]).double() * spread(w, ck.shape[1])


def close_checkpoint(ck, exp, want, E):
    """A checkpoint of values within E of `want`: the byte is the rule's for a
    maximum within E of the block's, each code half a step from its value."""
    a, top = block_max(want), block_max(E)
    s = torch.exp2(exp.double() - 127)
    assert bool(((a - top) <= 448 * s).all()) and bool(((2 * (a + top) > 448 * s) | (exp == 1) | (a == 0)).all())
    got, sc = load(ck, exp), spread(s, want.shape[1])
    lim = torch.maximum(R.U8[0] * want.abs(), R.SUB8[0] * sc) + (1 + R.U8[0]) * E
    bad = ~((got - want).abs() <= lim)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} kept values off, at {bad.nonzero()[0].tolist()}"


def forward(v, E, bias, act):
    """((g | u), bound), (h, bound) from the product of all 2F rows."""
    x = v if bias is None else v + bias.double()
    Ex = E + R.C * (v.abs() + (0 if bias is None else bias.double().abs()))
    F = v.shape[1] // 2
    g, u, Eg, Eu = x[:, :F], x[:, F:], Ex[:, :F], Ex[:, F:]
    a = R.act_of(g, act)
    Ea = 1.13 * Eg + (R.C * g.abs() if act else 0)      # every activation's slope is below 1.13
    h = a * u
    return (x, Ex), (h, u.abs() * Ea + (a.abs() + Ea) * Eu + R.C * h.abs())


def backward(v, E, x, act):
    """(dg | du) and its bound, from the product v of F rows and what was kept."""
    F = v.shape[1]
    g, u = x[:, :F].double(), x[:, F:].double()
    a, s = R.act_of(g, act), R.slope_of(g, act)
    d = torch.cat([v * u * s, v * a], 1)
    Ed = torch.cat([(u * s).abs() * E + R.C * (v * u).abs(), a.abs() * E + R.C * (v * g).abs()], 1)
    return d, Ed + R.C * d.abs()
