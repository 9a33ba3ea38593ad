"""fp8_block_norm and fp8_block_norm_bwd on more rows than run at once, so that each
workgroup goes through its row loop several times, the last time with rows past
the end: the next row's loads in flight, exchanges between wavefronts one row
after another, column sums over many rows."""
import pytest
import torch

import block_ref as R
from gpu_util import Guarded, say
from test_gpu_block_norm import BF, EPS, F32, inputs, ref_fwd, grads, setup_bwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from fp8_mixed_precision_linear_amd import lib
    return lib


# Columns: fewer than 8; a wavefront per row with one and with two vectors per
# lane; a workgroup per row with one, two and four vectors per thread.  Rows: the
# forward pass runs up to 8 workgroups of four rows, or of one, on each of 256
# compute units at once, the gradient one workgroup of up to 8 rows.
FORWARD = [(20011, 5), (20011, 136), (17001, 515), (18001, 1000), (5003, 1500), (5003, 2048), (3001, 4095), (3001, 8192),
           (2003, 9001), (2003, 16384), (1201, 20000), (1201, 32760)]


@pytest.mark.parametrize("shape", FORWARD)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("gate", ["channel", "full"])
def test_forward(L, shape, kind, stream, gate):
    rows, cols = shape
    layer, act = kind == "layer", rows % 3
    say("norm rows fwd", shape, kind, stream, gate)
    v = inputs(rows + cols, rows, cols, layer, stream, F32, gate, 0.5 if layer else 0.0)
    h, y, y8 = Guarded(shape, stream), Guarded(shape, BF), Guarded(shape, torch.uint8)
    # codes with each row's own scale, with one and an amax over all rows, or with one per 128 columns
    how, nb = "row" if gate == "full" else "tensor" if layer else "block", -(-cols // 128)
    sz, sh, amax = Guarded((rows, 2), F32), Guarded((rows, 2), F32), Guarded((1,), F32)
    si = Guarded((nb, rows) if how == "block" else (rows,), F32)
    amax.t.zero_()
    L.fp8_block_norm(v["x"], z=v["z"], h=h.t, y=y.t, kind=int(layer), eps=EPS, w_pre=v["w_pre"], b_pre=v["b_pre"], w_post=v["w_post"],
                     b_post=v["b_post"], gate=v["gate"], gate_act=act, res_scale=0.75, branch_scale=0.5, stats_z=sz.t, stats_h=sh.t, y8=y8.t,
                     y8_scaling={"row": L.SCALE_ROW, "tensor": L.SCALE_TENSOR, "block": L.SCALE_1x128}[how],
                     y8_scale_inv=None if how == "tensor" else si.t, y8_amax=amax.t if how == "tensor" else None,
                     y8_scale=torch.full((1,), 8.0, device="cuda") if how == "tensor" else None)
    torch.cuda.synchronize()
    for o in (h, y, y8, sz, sh, si, amax):
        o.check()
    r = ref_fwd(v, layer, act, 0.75, 0.5)
    R.close(h.t, r["h"], R.C * r["Sh"])
    R.close(y.t, r["y"], R.C * r["Sy"])
    spread = {"z": v["z"].double().abs().mean(1, keepdim=True), "h": r["Sh"].mean(1, keepdim=True)}
    for n, o in (("z", sz.t), ("h", sh.t)):
        m, q = r["stats_" + n][:, :1], r["stats_" + n][:, 1:]
        R.close(o[:, :1], m, R.C * spread[n])
        R.close(o[:, 1:], q, R.C * q * (1 + q * spread[n]))
    if how == "tensor":
        R.close(amax.t, r["y"].abs().max().reshape(1), R.C * r["Sy"].max())
        R.close8(y8.t, 0, r["y"] * 8, R.C * r["Sy"] * 8)
        return
    seg = cols if how == "row" else 128

    def most(t):   # over a row, or its segments: [segments][rows]
        pad = torch.zeros((rows, -(-cols // seg) * seg), dtype=torch.float64, device="cuda")
        pad[:, :cols] = t
        return pad.view(rows, -1, seg).amax(2).t()

    top, S = most(r["y"].abs()), most(r["Sy"])
    R.close(si.t.view(top.shape), top / 448, 3 * 2.0 ** -24 * top / 448 + R.C * S / 448)
    w = si.t.view(top.shape).double().t().repeat_interleave(seg, 1)[:, :cols]
    R.close8(y8.t, 0, r["y"] / w, R.C * r["Sy"] / w + 4 * 2.0 ** -24 * (r["y"] / w).abs())


# The gradient's column sums add at most 64 values one after the other: a lane's
# rows (20011 / 2048, 5003 / 1280 and fewer), up to 8 groups of a workgroup, 8
# parts, then 16.
BACKWARD = [(20011, 5), (9001, 136), (9001, 515), (9001, 1000), (5003, 1500), (5003, 2048), (3001, 4095), (2003, 8192), (1501, 9001),
            (1501, 16384), (1201, 20000), (1201, 32760)]


@pytest.mark.parametrize("shape", BACKWARD)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("stream", [BF, F32])
@pytest.mark.parametrize("gate", ["channel", "token", "full"])
def test_backward(L, shape, kind, stream, gate):
    rows, cols = shape
    layer, act, rs, bs = kind == "layer", cols % 3, 0.75, 0.5
    say("norm rows bwd", shape, kind, stream, gate)
    v, h, sh, sz, dy, dh, outs = setup_bwd(rows + cols, rows, cols, layer, stream, F32, gate, act, rs, bs)
    grads(L, v, layer, act, rs, bs, dy, dh, outs, h, sh, sz)
    torch.cuda.synchronize()
    want = R.norm_bwd(dy, dh, h, sh, v["z"], sz, layer, v["w_pre"], v["w_post"], v["b_post"], v["gate"], act, rs, bs)
    for n, o in outs.items():
        o.check()
        if n in ("db_pre", "db_post") and not layer:
            continue
        say(" ", n)
        R.close(o.t, want[n][0].reshape(o.t.shape), R.C * want[n][1].reshape(o.t.shape))


def test_no_columns(L):
    """The gradient of a gate per token is a sum over the columns: 0 without any."""
    x, g = torch.empty((70, 0), device="cuda"), torch.ones((70, 1), device="cuda")
    dg = Guarded((70, 1), F32)
    dg.t.fill_(5.0)
    L.fp8_block_norm_bwd(x, torch.empty_like(x), dh=x, z=x.to(BF), gate=g, dgate=dg.t, stats_z=torch.zeros((70, 2), device="cuda"))
    torch.cuda.synchronize()
    dg.check()
    assert bool((dg.t == 0).all())
    L.fp8_block_norm(x, z=x.to(BF), h=torch.empty_like(x), gate=g)   # and the pass itself has nothing to do
