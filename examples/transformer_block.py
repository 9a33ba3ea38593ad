"""One transformer block out of this library's calls: forward and backward of a
training step with delayed scaling, and the same block for single tokens.

    y0 = N(x)                           block norm -> FP8 codes and their amax
    q, k, v = y0 Wqkv^T                 FP8 linear;  q, k turned by fp8_rope
    a = attention(q, k, v) Wo^T         (the attention itself is the caller's)
    h = x + tanh(gate) * N(a)           block norm: gate, residual and the next
    y1 = N(h)                           block's norm in one pass
    u = gelu(y1 W1^T + b1)              FP8 linear: bias and activation on its
                                        way out, FP8 codes and their transpose
    out = h + u W2^T                    FP8 linear: residual on its way out

With --gated, u = silu(g) * w of (g | w) = y1 W1^T + b1 (W1 the gate's rows, then the up
projection's): one product, which keeps g | w for the backward pass in 8 bits; the
branch a is kept in 8 bits as well.

    python examples/transformer_block.py --tokens 4096 --hidden 4096 --ffn 14336 --heads 32 --kv-heads 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp8_mixed_precision_linear_amd import lib as L  # noqa: E402

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
T, ROW = L.SCALE_TENSOR, L.SCALE_ROW
EPS = 1e-6


def causal_attention(q, k, v):
    """Plain attention over one sequence, in float32."""
    q, k, v = (t.float().transpose(0, 1) for t in (q, k, v))
    rep = q.shape[0] // k.shape[0]
    k, v = k.repeat_interleave(rep, 0), v.repeat_interleave(rep, 0)
    s = torch.matmul(q, k.transpose(1, 2).contiguous()) * q.shape[2] ** -0.5
    n, m = s.shape[1:]
    s = s.masked_fill(torch.ones(n, m, dtype=torch.bool, device=s.device).triu(m - n + 1), float("-inf"))
    return torch.matmul(s.softmax(-1), v).transpose(0, 1).contiguous()


class Delayed:
    """Scales of tensors that are cast to one FP8 format, each from the amax of
    the steps before: scale, scale_inv and amax are views by name."""

    def __init__(self, names, fmt, device, length=16):
        self.fmt, n = fmt, len(names)
        self.history = torch.zeros(n, length, device=device)
        self.amax, self.scale, self.inv = torch.zeros(n, device=device), *torch.ones(2, n, device=device)
        self.at = {name: slice(i, i + 1) for i, name in enumerate(names)}

    def __getitem__(self, name):
        s = self.at[name]
        return self.scale[s], self.inv[s], self.amax[s]

    def step(self):
        L.fp8_amax_history_update_reset(self.history, self.amax, self.fmt, 0, L.AMAX_MAX, self.scale, self.inv)


class Weight:
    """E4M3 codes of w [out][in] and of its transpose, one scale."""

    def __init__(self, w):
        n, k = w.shape
        amax, self.scale, self.inv = torch.zeros(3, 1, device=w.device).unbind()
        L.fp8_amax(w, amax)
        L.fp8_compute_scale(amax, L.E4M3, 0, self.scale, self.inv)
        self.w = torch.empty(n, k, dtype=U8, device=w.device)
        self.t = torch.empty(k, n, dtype=U8, device=w.device)
        L.fp8_cast_amax_acc(w, L.E4M3, self.scale, amax, self.w, self.t)


class Block:
    def __init__(self, hidden, heads, kv_heads, head_dim, ffn, device="cuda", seed=0, gated=False):
        self.hidden, self.heads, self.kv, self.dim, self.ffn = hidden, heads, kv_heads, head_dim, ffn
        self.device, self.gated = device, gated
        self.first = first = 2 * ffn if gated else ffn      # rows of the feed-forward's first product
        g = torch.Generator(device="cpu").manual_seed(seed)

        def random(*shape, scale=1.0, mean=0.0):
            return (torch.randn(*shape, generator=g) * scale + mean).to(BF).to(device)

        wide = (heads + 2 * kv_heads) * head_dim
        self.param = {
            "wqkv": random(wide, hidden, scale=hidden ** -0.5),
            "wo": random(hidden, heads * head_dim, scale=(heads * head_dim) ** -0.5),
            "w1": random(first, hidden, scale=hidden ** -0.5),
            "w2": random(hidden, ffn, scale=ffn ** -0.5),
            "b1": random(first, scale=0.1), "gate": random(hidden, scale=0.5, mean=0.5),
            "n0": random(hidden, scale=0.1, mean=1.0), "n1": random(hidden, scale=0.1, mean=1.0),
            "na": random(hidden, scale=0.1, mean=1.0),
        }
        self.q8 = {n: Weight(self.param[n]) for n in ("wqkv", "wo", "w1", "w2")}
        self.act = Delayed(("y0", "o", "y1", "u"), L.E4M3, device)
        self.grad = Delayed(("out", "u", "a", "qkv"), L.E5M2, device)
        self.freqs = torch.empty(head_dim // 2, dtype=torch.float64, device=device)
        L.fp8_rope_freqs(self.freqs)

    def _new(self, *shape, dtype=BF):
        return torch.empty(*shape, dtype=dtype, device=self.device)

    def _split(self, qkv):
        t = qkv.view(qkv.shape[0], -1, self.dim)
        return t[:, :self.heads], t[:, self.heads:self.heads + self.kv], t[:, self.heads + self.kv:]

    def forward(self, x, positions=None, attend=causal_attention):
        """out [tokens][hidden], and what backward() needs (there the tokens are
        the inner dimension of products: a multiple of 16)."""
        p, q8, n = self.param, self.q8, x.shape[0]
        s = {"x": x, "positions": positions}
        # norm of the stream, cast on its way out
        s["y0"], y8 = self._new(n, self.hidden), self._new(n, self.hidden, dtype=U8)
        s["s0"] = self._new(n, 2, dtype=F32)
        scale, inv, amax = self.act["y0"]
        L.fp8_block_norm(x, y=s["y0"], eps=EPS, w_pre=p["n0"], stats_h=s["s0"], y8=y8, y8_scale=scale, y8_amax=amax)
        # queries, keys and values side by side; positions turned in place
        qkv = self._new(n, p["wqkv"].shape[0])
        L.fp8_scaled_gemm(y8, L.E4M3, T, inv, q8["wqkv"].w, L.E4M3, T, q8["wqkv"].inv, qkv)
        q, k, v = self._split(qkv)
        L.fp8_rope(q, self.freqs, positions, k)
        # attention, by autograd
        s["leaves"] = [t.detach().requires_grad_() for t in (q, k, v)]
        with torch.enable_grad():
            s["o_graph"] = attend(*s["leaves"])
        o = s["o_graph"].detach().to(BF).view(n, -1)
        o8, s["o8_t"] = self._new(*o.shape, dtype=U8), self._new(*o.shape[::-1], dtype=U8)
        scale, inv, amax = self.act["o"]
        L.fp8_cast_amax_acc(o, L.E4M3, scale, amax, o8, s["o8_t"])
        s["a"] = self._new(n, self.hidden)
        L.fp8_scaled_gemm(o8, L.E4M3, T, inv, q8["wo"].w, L.E4M3, T, q8["wo"].inv, s["a"])
        # the branch back into the stream, and the next norm
        s["h"], s["y1"] = self._new(n, self.hidden), self._new(n, self.hidden)
        y8 = self._new(n, self.hidden, dtype=U8)
        s["sa"], s["s1"] = self._new(n, 2, dtype=F32), self._new(n, 2, dtype=F32)
        scale, inv, amax = self.act["y1"]
        L.fp8_block_norm(x, s["a"], s["h"], s["y1"], eps=EPS, w_pre=p["n1"], w_post=p["na"], gate=p["gate"],
                         gate_act=L.GATE_TANH, stats_z=s["sa"], stats_h=s["s1"], y8=y8, y8_scale=scale, y8_amax=amax)
        # the feed-forward pair
        u8, s["u8_t"] = self._new(n, self.ffn, dtype=U8), self._new(self.ffn, n, dtype=U8)
        uscale, uinv, uamax = self.act["u"]
        written = dict(bias=p["b1"], d_scale=uscale, d_fmt=L.E4M3, D_t=s["u8_t"], d_amax=uamax, amax_accumulate=True)
        if self.gated:
            s["kept"] = self._checkpoint(n, self.ffn, 2)
            L.fp8_gated_linear(y8, L.E4M3, T, inv, q8["w1"].w, L.E4M3, T, q8["w1"].inv, u8, act=L.ACT_SILU,
                               ck=s["kept"][0], ck_exp=s["kept"][1], **written)
            s["a8"] = self._checkpoint(n, self.hidden)
            L.fp8_checkpoint_save(s.pop("a"), *s["a8"])
        else:
            s["aux"] = self._new(n, self.ffn)
            L.fp8_scaled_gemm_ep(y8, L.E4M3, T, inv, q8["w1"].w, L.E4M3, T, q8["w1"].inv, u8, act=L.ACT_GELU,
                                 aux=s["aux"], **written)
        out = self._new(n, self.hidden)
        L.fp8_scaled_gemm_ep(u8, L.E4M3, T, uinv, q8["w2"].w, L.E4M3, T, q8["w2"].inv, out, residual=s["h"])
        # the scales that this step's codes were made with (step() changes them in place)
        s["inv"] = {name: self.act[name][1].clone() for name in self.act.at}
        s["scale"] = {name: self.act[name][0].clone() for name in self.act.at}
        return out, s

    def _checkpoint(self, rows, cols, parts=1):
        """Room for an 8-bit checkpoint of `parts` matrices side by side: codes, powers of two."""
        return self._new(rows, parts * cols, dtype=U8), self._new(rows, parts * ((cols + 31) // 32), dtype=U8)

    def _cast(self, g, name):
        """E5M2 codes of a gradient and of its transpose, and their inverse scale."""
        c, t = self._new(*g.shape, dtype=U8), self._new(*g.shape[::-1], dtype=U8)
        scale, inv, amax = self.grad[name]
        L.fp8_cast_amax_acc(g, L.E5M2, scale, amax, c, t)
        return c, t, inv

    def _wgrad(self, g8_t, ginv, y8_t, yinv):
        dw = self._new(g8_t.shape[0], y8_t.shape[0], dtype=F32)
        L.fp8_scaled_gemm(g8_t, L.E5M2, T, ginv, y8_t, L.E4M3, T, yinv, dw)
        return dw

    def _transposed(self, y, scale):
        """E4M3 codes [cols][rows] of an activation kept in bf16 (the norm writes
        its codes row by row only, so a weight gradient's operand is a cast of its own)."""
        t = self._new(*y.shape[::-1], dtype=U8)
        L.fp8_cast_amax_acc(y, L.E4M3, scale, torch.zeros(1, device=self.device), None, t)
        return t

    def backward(self, dout, s):
        """(dx, {parameter: gradient})"""
        p, q8, n, g = self.param, self.q8, dout.shape[0], {}
        # feed-forward: the second product's gradient runs through the first's
        # activation on its way out, with the bias gradient
        d8, d8_t, dinv = self._cast(dout, "out")
        g["w2"] = self._wgrad(d8_t, dinv, s["u8_t"], s["inv"]["u"])
        u8, u8_t = self._new(n, self.first, dtype=U8), self._new(self.first, n, dtype=U8)
        g["b1"] = torch.empty_like(p["b1"])
        uscale, uinv, uamax = self.grad["u"]
        written = dict(backward=True, dbias=g["b1"], d_scale=uscale, d_fmt=L.E5M2, D_t=u8_t, d_amax=uamax,
                       amax_accumulate=True)
        if self.gated:
            L.fp8_gated_linear(d8, L.E5M2, T, dinv, q8["w2"].t, L.E4M3, T, q8["w2"].inv, u8, act=L.ACT_SILU,
                               ck=s["kept"][0], ck_exp=s["kept"][1], **written)
            a = self._new(n, self.hidden)
            L.fp8_checkpoint_load(*s["a8"], a)
        else:
            a = s["a"]
            L.fp8_scaled_gemm_ep(d8, L.E5M2, T, dinv, q8["w2"].t, L.E4M3, T, q8["w2"].inv, u8, act=L.ACT_GELU,
                                 aux=s["aux"], **written)
        g["w1"] = self._wgrad(u8_t, uinv, self._transposed(s["y1"], s["scale"]["y1"]), s["inv"]["y1"])
        dy = self._new(n, self.hidden)
        L.fp8_scaled_gemm(u8, L.E5M2, T, uinv, q8["w1"].t, L.E4M3, T, q8["w1"].inv, dy)
        # both norms, the gate and the residual in one pass
        dx, da = self._new(n, self.hidden), self._new(n, self.hidden)
        g["n1"], g["na"], g["gate"] = (torch.empty_like(p["n1"]) for _ in range(3))
        L.fp8_block_norm_bwd(s["h"], dx, dy=dy, dh=dout, z=a, dz=da, w_pre=p["n1"], w_post=p["na"],
                             gate=p["gate"], gate_act=L.GATE_TANH, stats_z=s["sa"], stats_h=s["s1"],
                             dw_pre=g["n1"], dw_post=g["na"], dgate=g["gate"])
        # attention
        a8, a8_t, ainv = self._cast(da, "a")
        g["wo"] = self._wgrad(a8_t, ainv, s["o8_t"], s["inv"]["o"])
        do = self._new(n, self.heads * self.dim)
        L.fp8_scaled_gemm(a8, L.E5M2, T, ainv, q8["wo"].t, L.E4M3, T, q8["wo"].inv, do)
        dqkv = self._new(n, p["wqkv"].shape[0])
        for view, grad in zip(self._split(dqkv), torch.autograd.grad(s["o_graph"], s["leaves"],
                                                                     do.view(s["o_graph"].shape).float())):
            view.copy_(grad)
        dq, dk, _ = self._split(dqkv)
        L.fp8_rope(dq, self.freqs, s["positions"], dk, inverse=True)
        c8, c8_t, cinv = self._cast(dqkv, "qkv")
        g["wqkv"] = self._wgrad(c8_t, cinv, self._transposed(s["y0"], s["scale"]["y0"]), s["inv"]["y0"])
        L.fp8_scaled_gemm(c8, L.E5M2, T, cinv, q8["wqkv"].t, L.E4M3, T, q8["wqkv"].inv, dy)
        g["n0"] = torch.empty_like(p["n0"])
        L.fp8_block_norm_bwd(s["x"], dx, dy=dy, dh=dx, w_pre=p["n0"], stats_h=s["s0"], dw_pre=g["n0"])
        return dx, g

    def step(self):
        """The step's amax values become the next one's scales."""
        self.act.step()
        self.grad.step()

    def decode(self, x, position, cache_k, cache_v, attend=causal_attention):
        """out of tokens that follow the cache's [position] ones: activations
        scaled row by row, so that no token's codes depend on another's."""
        p, q8, n = self.param, self.q8, x.shape[0]
        y8, inv = self._new(n, self.hidden, dtype=U8), self._new(n, dtype=F32)
        L.fp8_block_norm(x, eps=EPS, w_pre=p["n0"], y8=y8, y8_scaling=ROW, y8_scale_inv=inv)
        qkv = self._new(n, p["wqkv"].shape[0])
        L.fp8_scaled_gemm_ep(y8, L.E4M3, ROW, inv, q8["wqkv"].w, L.E4M3, T, q8["wqkv"].inv, qkv)
        q, k, v = self._split(qkv)
        k_new = cache_k[position:position + n]
        L.fp8_rope(q, self.freqs, None, k, k_out=k_new, offset=position)   # keys straight into the cache
        cache_v[position:position + n].copy_(v)
        o = attend(q, cache_k[:position + n], cache_v[:position + n]).to(BF).view(n, -1)
        o8 = self._new(*o.shape, dtype=U8)
        L.fp8_cast_rowwise(o, L.E4M3, o8, inv)
        a = self._new(n, self.hidden)
        L.fp8_scaled_gemm_ep(o8, L.E4M3, ROW, inv, q8["wo"].w, L.E4M3, T, q8["wo"].inv, a)
        h = self._new(n, self.hidden)
        L.fp8_block_norm(x, a, h, eps=EPS, w_pre=p["n1"], w_post=p["na"], gate=p["gate"], gate_act=L.GATE_TANH,
                         y8=y8, y8_scaling=ROW, y8_scale_inv=inv)
        u = self._new(n, self.ffn)
        first, act = (L.fp8_gated_linear, L.ACT_SILU) if self.gated else (L.fp8_scaled_gemm_ep, L.ACT_GELU)
        first(y8, L.E4M3, ROW, inv, q8["w1"].w, L.E4M3, T, q8["w1"].inv, u, bias=p["b1"], act=act)
        u8 = self._new(n, self.ffn, dtype=U8)
        L.fp8_cast_rowwise(u, L.E4M3, u8, inv)
        out = self._new(n, self.hidden)
        L.fp8_scaled_gemm_ep(u8, L.E4M3, ROW, inv, q8["w2"].w, L.E4M3, T, q8["w2"].inv, out, residual=h)
        return out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 1024), ("hidden", 2048), ("heads", 16), ("kv-heads", 4), ("ffn", 8192),
                        ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--gated", action="store_true")
    a = ap.parse_args()
    b = Block(a.hidden, a.heads, a.kv_heads, a.hidden // a.heads, a.ffn, gated=a.gated)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(BF)
    dout = torch.randn(a.tokens, a.hidden, device="cuda").to(BF)

    def train():
        out, s = b.forward(x)
        b.backward(dout, s)
        b.step()
        return out

    def timed(what, fn):
        for _ in range(3):
            fn()
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(a.steps):
            fn()
        stop.record()
        torch.cuda.synchronize()
        print(f"{what}: {start.elapsed_time(stop) / a.steps:.3f} ms", flush=True)

    timed(f"forward + backward, {a.tokens} tokens", train)
    ck, cv = (torch.zeros(a.tokens + 1, a.kv_heads, b.dim, device="cuda", dtype=BF) for _ in range(2))
    timed("one token", lambda: b.decode(x[:1], a.tokens, ck, cv))


if __name__ == "__main__":
    main()
