"""Plain 64-bit forms of the operators around the linears (norms with gate and
residual scale, the GEMM with the linear's epilogue, rotary positions) and the
error bounds that their kernels are held to.

The bounds count roundings.  u(t) = eps / 2 is the relative error of one
rounding to type t.  The kernels' arithmetic is binary32; a result that comes
out of at most ~60 chained binary32 operations on terms whose magnitudes add up
to S is within C * S of the exact one, C = 64 * 2^-24 (row sums: at most 32
values per thread one after the other, then a tree; rsqrt, exp and rcp within
2 units).  S is carried along beside every value."""
import math

import torch

C = 64 * 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FMAX = (448.0, 57344.0)
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
U8 = (2.0 ** -4, 2.0 ** -3)
SUB8 = (2.0 ** -10, 2.0 ** -17)   # half the step of the format's subnormals


def d(t):
    return None if t is None else t.double()


def close(got, want, slack, dtype=None):
    """|got - want| <= u |want| + slack, elementwise (u: of got's type)."""
    u = U[dtype or got.dtype]
    err = (got.double() - want).abs()
    lim = u * want.abs() + (1 + u) * slack + 2.0 ** -133
    bad = ~(err <= lim)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} off: worst {float((err / lim).max()):.3g} times its bound, at "
        f"{bad.nonzero()[0].tolist()}: {float(got.double()[bad][0])} for {float(want[bad][0])}")


def close8(codes, fmt, want, slack):
    """Codes within half a step of the scaled value `want` (saturating)."""
    got = codes.view(F8[fmt]).double()
    w = want.clamp(-FMAX[fmt], FMAX[fmt])
    lim = torch.clamp(U8[fmt] * w.abs(), min=SUB8[fmt]) + (1 + U8[fmt]) * slack
    bad = ~((got - w).abs() <= lim)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} codes off, at {bad.nonzero()[0].tolist()}: "
        f"{float(got[bad][0])} for {float(w[bad][0])}")


# ---- norm

def gate_of(g, act):
    if g is None:
        return None
    g = g.double()
    return torch.sigmoid(g) if act == 1 else torch.tanh(g) if act == 2 else g


def stats(v, layer, eps):
    m = v.mean(1, keepdim=True) if layer else torch.zeros_like(v[:, :1])
    r = 1 / torch.sqrt(((v - m) ** 2).mean(1, keepdim=True) + eps)
    return m, r


def norm_fwd(x, z, layer, eps, w_pre=None, b_pre=None, w_post=None, b_post=None, gate=None, gate_act=0,
             res_scale=1.0, branch_scale=1.0):
    """{h, y, stats} in 64 bits, and the magnitudes S of h and y."""
    one = torch.ones(x.shape[1], dtype=torch.float64, device=x.device)
    wpre, wpost = (one if w is None else w.double() for w in (w_pre, w_post))
    bpre, bpost = (0 * one if b is None else b.double() for b in (b_pre, b_post))
    h = x.double()
    S = h.abs()
    r = {}
    if z is not None:
        zz = z.double()
        m, rs = stats(zz, layer, eps)
        g = gate_of(gate, gate_act)
        g = torch.ones((), dtype=torch.float64, device=x.device) if g is None else g
        n = (zz - m) * rs * wpost + bpost
        h = res_scale * h + branch_scale * g * n
        spread = zz.abs() + zz.abs().mean(1, keepdim=True)
        S = abs(res_scale) * S + abs(branch_scale) * g.abs() * (spread * rs * wpost.abs() + bpost.abs())
        r["stats_z"] = torch.cat([m, rs], 1)
    m, rs = stats(h, layer, eps)
    r["y"] = (h - m) * rs * wpre + bpre
    r["Sy"] = rs * wpre.abs() * (S + S.mean(1, keepdim=True) + h.abs() * (1 + rs * S.mean(1, keepdim=True))) + bpre.abs()
    r["h"], r["Sh"] = h, S
    r["stats_h"] = torch.cat([m, rs], 1)
    return r


def _norm_back(dd, Sd, v, st, w, layer):
    """Gradient of a norm's input from that of its output, and its magnitude."""
    m, r = st[:, :1].double(), st[:, 1:].double()
    xh = (v - m) * r
    Sx = (v.abs() + m.abs()) * r
    a, Sa = dd * w, Sd * w.abs()
    t = a - xh * (a * xh).mean(1, keepdim=True)
    S = Sa + Sx * (Sa * Sx).mean(1, keepdim=True)
    if layer:
        t = t - a.mean(1, keepdim=True)
        S = S + Sa.mean(1, keepdim=True)
    return t * r, S * r, xh, Sx


def norm_bwd(dy, dh, h, stats_h, z, stats_z, layer, w_pre=None, w_post=None, b_post=None, gate=None, gate_act=0,
             res_scale=1.0, branch_scale=1.0):
    """Gradients by the formulas, {name: (value, magnitude)}."""
    base = h
    one = torch.ones(base.shape[1], dtype=torch.float64, device=base.device)
    wpre, wpost = (one if w is None else w.double() for w in (w_pre, w_post))
    r = {}
    dH = torch.zeros(base.shape, dtype=torch.float64, device=base.device) if dh is None else dh.double()
    S = dH.abs()
    if dy is not None:
        dyd = dy.double()
        t, St, xh, Sx = _norm_back(dyd, dyd.abs(), h.double(), stats_h, wpre, layer)
        dH, S = dH + t, S + St
        r["dw_pre"] = (dyd * xh).sum(0), (dyd.abs() * Sx).sum(0)
        r["db_pre"] = dyd.sum(0), dyd.abs().sum(0)
    r["dx"] = (dH, S) if z is None else (res_scale * dH, abs(res_scale) * S)
    if z is not None:
        g = gate_of(gate, gate_act)
        gv = torch.ones((), dtype=torch.float64, device=base.device) if g is None else g
        dn, Sn = branch_scale * gv * dH, abs(branch_scale) * gv.abs() * S
        dz, Sz, zh, Szh = _norm_back(dn, Sn, z.double(), stats_z, wpost, layer)
        r["dz"] = dz, Sz
        r["dw_post"] = (dn * zh).sum(0), (Sn * Szh).sum(0)
        r["db_post"] = dn.sum(0), Sn.sum(0)
        if g is not None:
            slope = g * (1 - g) if gate_act == 1 else 1 - g * g if gate_act == 2 else torch.ones_like(g)
            b = 0 * one if b_post is None else b_post.double()
            n, Sv = zh * wpost + b, Szh * wpost.abs() + b.abs()
            dg, Sg = branch_scale * dH * n * slope, abs(branch_scale) * S * Sv
            if gate.dim() == 1:
                dg, Sg = dg.sum(0), Sg.sum(0)
            elif gate.shape[1] == 1 and base.shape[1] != 1:
                dg, Sg = dg.sum(1, keepdim=True), Sg.sum(1, keepdim=True)
            r["dgate"] = dg, Sg
    return r


# ---- linear

def act_of(u, act):
    F = torch.nn.functional
    return (u, F.relu(u), F.gelu(u), F.gelu(u, approximate="tanh"), F.silu(u))[act]


def slope_of(u, act):
    u = u.detach().clone().requires_grad_()
    return torch.autograd.grad(act_of(u, act).sum(), u)[0] if act else torch.ones_like(u)


def wide(codes, fmt, sinv, scaling):
    """Dequantised operand [rows][K] in 64 bits."""
    x = codes.view(F8[fmt]).double()
    s = sinv.double()
    if scaling == 0:
        return x * s
    if scaling == 5:
        return x * s[:, None]
    seg = s.t().repeat_interleave(128, 1)
    return x * (seg if scaling in (1, 3) else seg.repeat_interleave(128, 0)[:x.shape[0]])


def product(A, af, asc, sa, B, bf, bsc, sb):
    """v = A B^T and the bound on the matrix unit's value of it: each product of
    a group of 8 loses less than 2^-13 of the group's largest (all of it at
    most 8 * 2^-13 of the group's sum of magnitudes), and the groups are
    combined, scaled and added in binary32."""
    a, b = wide(A, af, sa, asc), wide(B, bf, sb, bsc)
    v, D = a @ b.t(), a.abs() @ b.abs().t()
    return v, (8 * 2.0 ** -13 + (A.shape[1] / 8 + 16) * 2.0 ** -23) * D


def linear_fwd(v, E, bias, act, residual, res_scale):
    """(u, bound), (d, bound): every activation's slope is below 1.13, its own
    arithmetic is within C of |u|."""
    u = v if bias is None else v + bias.double()
    Eu = E + C * (v.abs() + (0 if bias is None else bias.double().abs()))
    o = act_of(u, act)
    Eo = 1.13 * Eu + (C * u.abs() if act else 0)
    if residual is not None:
        o = o + res_scale * residual.double()
        Eo = Eo + C * (o.abs() + abs(res_scale) * residual.double().abs())
    return (u, Eu), (o, Eo)


def linear_bwd(v, E, aux, act):
    s = slope_of(aux.double(), act) if act else torch.ones_like(v)
    o = v * s
    return o, s.abs() * E + C * v.abs()


# ---- rope

def rope(x, pos, freqs, interleaved, inverse, scale):
    n = freqs.numel()
    a = pos.double()[:, None, None] * freqs
    c, s = scale * a.cos(), scale * a.sin() * (-1 if inverse else 1)
    out = x.double().clone()
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x0, x1 = x[..., lo].double(), x[..., hi].double()
    out[..., lo], out[..., hi] = x0 * c - x1 * s, x1 * c + x0 * s
    S = torch.zeros_like(out)
    S[..., lo] = S[..., hi] = abs(scale) * (x0.abs() + x1.abs())
    return out, S


def rope_freqs(pairs, base, scaling, factor, trained, low, high):
    if scaling == 2 and pairs > 1:
        base *= factor ** (pairs / (pairs - 1))
    f = torch.tensor([base ** (-i / pairs) for i in range(pairs)], dtype=torch.float64)
    if scaling == 1:
        f = f / factor
    if scaling == 3:
        keep = ((trained * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f
