"""Infinities in the backward call of fp8_gated_linear: what the outputs do not have, the rows
and columns past the last ones of a tile, adds nothing to the amax or to the bias gradients (an
infinity times the zeros that stand there is a NaN).  On each kernel; every value is positive,
so an infinity stays one."""
import pytest
import torch

import gated_ref as G
from gpu_util import Guarded, say
from test_gpu_gated import FEW, LARGE, TILES, L, taken      # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
INF = float("inf")

# rows, outputs, K, scalings of A and B, kernel, rows of its tiles, whether K is cut; the large tiles'
# last columns are 32 of 256, their last rows 4 of 256
PATHS = [
    (5, 203, 256, (5, 0), FEW, 16, False), (40, 203, 256, (5, 0), TILES, 32, False), (64, 520, 8192, (5, 0), TILES, 32, True),
    (1037, 1999, 2320, (5, 5), TILES, 64, False), (1500, 4095, 656, (5, 0), TILES, 128, False),
    (2052, 4128, 640, (5, 0), LARGE, 256, False), (2052, 4128, 656, (5, 5), LARGE, 256, False),
    (2052, 4128, 640, (1, 2), LARGE, 256, False), (2052, 4128, 640, (3, 4), LARGE, 256, False)]


def operand(g, rows, K, codes, scaling):
    """Codes drawn from `codes`, and inverse scales of 1 for that scaling."""
    t = torch.tensor(codes, dtype=U8, device="cuda")[torch.randint(0, len(codes), (rows, K), generator=g, device="cuda")]
    nkb, nrb = -(-K // 128), -(-rows // 128)
    shape = {0: (1,), 5: (rows,), 1: (nkb, rows), 3: (nkb, rows)}.get(scaling, (nkb, nrb))
    return t, torch.ones(shape, device="cuda")


def call(L, path, kept, out, change):
    """(D, amax, dbias) of a backward call whose gradient and scales `change` has made infinite somewhere."""
    M, F, K, (asc, bsc) = path[:4]
    g = torch.Generator(device="cuda").manual_seed(M + F)
    A, sa = operand(g, M, K, [0x38, 0x3C], asc)       # E5M2: 0.5, 1
    B, sb = operand(g, F, K, [0x30, 0x38], bsc)                          # E4M3: 0.5, 1
    change(A, sa, sb)
    x = 1 + torch.randint(0, 2, (M, 2 * F), generator=g, device="cuda").float()
    kw = dict(act=L.ACT_RELU, backward=True)
    if kept == "bf16":
        kw["aux"] = x.to(BF)
    else:
        kw["ck"], kw["ck_exp"] = (torch.cat(t, 1) for t in zip(G.save(x[:, :F]), G.save(x[:, F:])))
    D, amax, db = Guarded((M, 2 * F), BF if out == "bf16" else U8), Guarded((1,), F32), Guarded((2 * F,), F32)
    if out == "e5m2":
        kw.update(d_fmt=L.E5M2, d_scale=torch.ones(1, device="cuda"))
    say("gated infinity", path, kept, out)
    L.fp8_gated_linear(A, L.E5M2, asc, sa, B, L.E4M3, bsc, sb, D.t, d_amax=amax.t, dbias=db.t, **kw)
    torch.cuda.synchronize()
    for t in (D, amax, db):
        t.check()
    return D.t, float(amax.t), db.t


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("kept", ["bf16", "ckpt"])
@pytest.mark.parametrize("out", ["bf16", "e5m2"])
def test_infinite_gradient(L, taken, path, kept, out):
    """One infinity among a token's gradients: its row is infinite, and so are the amax and every sum."""
    at = path[0] // 2

    def change(A, sa, sb):
        A[at, 100] = 0x7C
    D, amax, db = call(L, path, kept, out, change)
    others = torch.arange(path[0], device="cuda") != at
    if out == "bf16":
        assert bool((D[at] == INF).all()) and bool(D[others].isfinite().all())
    else:
        assert bool((D[at] == 0x7B).all())          # the format's largest
    assert amax == INF
    assert int((db == INF).sum()) == db.numel()
    assert taken == [path[4:7]]


@pytest.mark.parametrize("path", [p for p in PATHS if p[3][0] == 5])
@pytest.mark.parametrize("kept", ["bf16", "ckpt"])
@pytest.mark.parametrize("out", ["bf16", "e5m2"])
def test_infinite_scale_of_the_last_row(L, taken, path, kept, out):
    """The rows past the last have no scale of their own."""
    def change(A, sa, sb):
        sa[-1] = INF
    D, amax, db = call(L, path, kept, out, change)
    if out == "bf16":
        assert bool((D[-1] == INF).all()) and bool(D[:-1].isfinite().all())
    else:
        assert bool((D[-1] == 0x7B).all())
    assert amax == INF
    assert int((db == INF).sum()) == db.numel()
    assert taken == [path[4:7]]


@pytest.mark.parametrize("path", [p for p in PATHS if p[3][1] != 4])      # (powers of two are finite)
@pytest.mark.parametrize("kept", ["bf16", "ckpt"])
@pytest.mark.parametrize("out", ["bf16", "e5m2"])
def test_infinite_scale_of_weights(L, taken, path, kept, out):
    """Of all of them, of one column or of one block's: its columns are infinite, and their sums."""
    F, bsc = path[1], path[3][1]
    bad = torch.zeros(F, dtype=torch.bool, device="cuda")
    bad[slice(None) if bsc == 0 else slice(7, 8) if bsc == 5 else slice(128, 256)] = True
    bad = bad.repeat(2)

    def change(A, sa, sb):
        if bsc in (2, 4):
            sb[1, 1] = INF
        else:
            sb[7 if bsc == 5 else 0] = INF
    D, amax, db = call(L, path, kept, out, change)
    if out == "bf16":
        assert bool((D[:, bad] == INF).all()) and bool(D[:, ~bad].isfinite().all())
    else:
        assert bool((D[:, bad] == 0x7B).all())
    assert amax == INF
    assert int((db[bad] == INF).sum()) == int(bad.sum()) and bool(db[~bad].isfinite().all())
    assert taken == [path[4:7]]
