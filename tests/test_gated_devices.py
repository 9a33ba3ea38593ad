"""The gated pair and the checkpoints refuse a tensor, or a stream, of another GPU than the current
one before anything is launched: the kernel would go to the current one and read the other's memory.
Host memory stands in for two GPUs, and nothing is launched (these run without one)."""
import pytest
import torch

U8, BF, F32 = torch.uint8, torch.bfloat16, torch.float32


class OnGpu(torch.Tensor):
    """A tensor that says it is on GPU `where`."""
    where, is_cuda = 0, True

    def get_device(self):
        return self.where


@pytest.fixture
def L(monkeypatch):
    from fp8_mixed_precision_linear_amd import lib
    lib.launched = launched = []

    def call(*a):
        launched.append(a)
        return 0
    for name in ("fp8_gated_linear", "fp8_checkpoint_save", "fp8_checkpoint_load"):
        monkeypatch.setattr(lib._L, name, call)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    yield lib
    del lib.launched


def gpu(shape, dtype, where=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)
    t.where = where
    return t


M, F, K = 4, 40, 128


def forward(L, at):
    t = {n: gpu(shape, dt, 1 if n == at or at == "all" else 0) for n, (shape, dt) in dict(
        A=((M, K), U8), sa=((1,), F32), B=((2 * F, K), U8), sb=((1,), F32), D=((M, F), U8), bias=((2 * F,), F32), aux=((M, 2 * F), BF),
        ck=((M, 2 * F), U8), ck_exp=((M, 4), U8), d_amax=((1,), F32), d_scale=((1,), F32), D_t=((F, M), U8),
        workspace=((1 << 16,), U8)).items()}
    a = [t.pop(n) for n in ("A", "sa", "B", "sb", "D")]
    L.fp8_gated_linear(a[0], 0, 0, a[1], a[2], 0, 0, a[3], a[4], d_fmt=0, **t)


def backward(L, at):
    t = {n: gpu(shape, dt, 1 if n == at or at == "all" else 0) for n, (shape, dt) in dict(
        A=((M, K), U8), sa=((1,), F32), B=((F, K), U8), sb=((1,), F32), D=((M, 2 * F), BF), aux=((M, 2 * F), BF), dbias=((2 * F,), BF),
        workspace=((1 << 16,), U8)).items()}
    a = [t.pop(n) for n in ("A", "sa", "B", "sb", "D")]
    L.fp8_gated_linear(a[0], 1, 0, a[1], a[2], 0, 0, a[3], a[4], backward=True, **t)


def checkpoint(call, strided):
    def run(L, at):
        x, ck, exp = (gpu(s, dt, 1 if n == at or at == "all" else 0) for n, s, dt in (("x", (M, F + 1), F32), ("ck", (M, F + 1), U8),
                                                                                    ("exp", (M, 3), U8)))
        if strided:
            x, ck, exp = x[:, :F], ck[:, :F], exp[:, :2]
            for t, n in ((x, "x"), (ck, "ck"), (exp, "exp")):
                t.where = 1 if n == at or at == "all" else 0
        else:
            exp = exp[:, :2].contiguous()
            exp.where = 1 if at in ("exp", "all") else 0
        if call == "save":
            L.fp8_checkpoint_save(x, ck, exp)
        else:
            L.fp8_checkpoint_load(ck, exp, x)
    return run


CALLS = [(forward, ["A", "sa", "B", "sb", "D", "bias", "aux", "ck", "ck_exp", "d_amax", "d_scale", "D_t", "workspace"]),
         (backward, ["A", "sa", "B", "sb", "D", "aux", "dbias", "workspace"])]
CALLS += [(checkpoint(c, s), ["x", "ck", "exp"]) for c in ("save", "load") for s in (False, True)]


@pytest.mark.parametrize("call,tensors", CALLS)
def test_tensor_of_another_device(L, call, tensors):
    call(L, None)
    assert len(L.launched) == 1
    for at in tensors + ["all"]:
        with pytest.raises(ValueError):
            call(L, at)
    assert len(L.launched) == 1


def test_stream_of_another_device(L, monkeypatch):
    class Stream:
        device_index, cuda_stream = 1, 7
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    x, ck, exp = gpu((M, F), F32), gpu((M, F), U8), gpu((M, 2), U8)
    with pytest.raises(ValueError):
        L.fp8_checkpoint_save(x, ck, exp, stream=Stream())
    assert not L.launched
    Stream.device_index = 0
    L.fp8_checkpoint_save(x, ck, exp, stream=Stream())
    assert L.launched[0][-1] == 7
