"""Refusals of the gated half: every call below fails a host-side check, so nothing is launched
and no GPU is needed."""
import ctypes

import pytest
import torch

import kronecker_factored_structured_b200 as kfs
from kronecker_factored_structured_b200 import native

V = ctypes.c_void_p
OK, ODD = V(0x10000), V(0x10008)           # never dereferenced
GX, GS, GA, GB, Gb, OUT = (V(0x20000 + 0x1000 * i) for i in range(6))


def call(backward, x=OK, S=OK, A=OK, B=OK, bias=OK, h=OUT, dX=GX, dS=GS, dA=GA, dB=GB, dbias=Gb,
         N=8, p=4, q=4, m1=16, m2=16, r=2, act=0, dtype=2, flags=0, ws=OK, ws_bytes=1 << 40):
    lib = native.load()
    tail = (N, p, q, m1, m2, r, act, dtype, flags, ws, ws_bytes, None)
    if backward:
        return lib.kron_glu_backward(x, S, A, B, bias, h, dX, dS, dA, dB, dbias, *tail)
    return lib.kron_glu_forward(x, S, A, B, bias, h, *tail)


COMMON = [(dict(dtype=3), 1), (dict(dtype=1), 2), (dict(act=-1), 1), (dict(act=4), 1),
          (dict(flags=1), 1), (dict(N=-1), 1), (dict(N=(1 << 30) + 1), 1), (dict(p=0), 1),
          (dict(q=0), 1), (dict(r=0), 1), (dict(m1=0), 1), (dict(m1=12), 2), (dict(m2=4), 2),
          (dict(m1=6, dtype=0), 2), (dict(p=1 << 20), 1), (dict(r=2000), 1), (dict(p=1025), 2),
          (dict(p=64, q=64, m1=64, m2=64, r=100), 2),
          (dict(p=4096, q=4096, m1=256, m2=256, r=64, dtype=0), 2),
          (dict(x=None), 1), (dict(S=None), 1), (dict(A=None), 1), (dict(B=None), 1),
          (dict(h=None), 1), (dict(x=ODD), 3), (dict(bias=ODD), 3), (dict(h=ODD), 3),
          (dict(S=None, N=0), 1)]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kwargs,status", COMMON)
def test_rejects(backward, kwargs, status):
    assert call(backward, **kwargs) == status
    assert native.load().kron_last_error().decode() != ""


@pytest.mark.parametrize("kwargs,status", [
    (dict(dS=None), 1), (dict(dA=None), 1), (dict(dB=None), 1), (dict(dX=ODD), 3),
    (dict(dbias=ODD), 3), (dict(dX=OK), 1), (dict(dS=OK), 1), (dict(dA=OK), 1), (dict(dB=OK), 1),
    (dict(dbias=OK), 1), (dict(ws=None), 4), (dict(ws_bytes=100), 4), (dict(ws=V(0x10010)), 3)])
@pytest.mark.parametrize("dtype", [0, 2])
def test_backward_rejects(dtype, kwargs, status):
    assert call(True, dtype=dtype, **kwargs) == status


def test_forward_is_not_in_place():
    assert call(False, h=OK) == 1


def test_forward_f32_wants_its_workspace():
    """The compiled shape over many rows goes through one pre-activation in memory."""
    big = dict(dtype=0, N=4096, p=32, q=32, m1=32, m2=32, r=4)
    assert native.glu_workspace_size(4096, 32, 32, 32, 32, 4, "f32") == 4096 * 1024 * 4
    assert call(False, ws=None, **big) == 4
    assert call(False, ws_bytes=4096, **big) == 4
    assert call(False, ws=V(0x10010), **big) == 3


def test_empty_forward_is_fine():
    assert call(False, N=0, x=None, h=None, ws=None, ws_bytes=0) == 0


def test_workspace_size():
    size = native.glu_workspace_size
    assert size(100, 4, 4, 16, 16, 2, "bf16") == 0            # the forward needs none
    assert size(100, 4, 4, 16, 16, 2, "f32") == 0             # one kernel
    for dt in ("f32", "bf16"):
        n = size(100, 4, 4, 16, 16, 2, dt, True)
        assert n > 0 and n == size(100, 4, 4, 16, 16, 2, dt, True)
    assert size(100, 4, 4, 16, 16, 2, "tf32", True) == 0
    assert size(0, 4, 4, 16, 16, 2, "bf16", True) == 0


def test_every_shape_of_a_wide_range_has_a_kernel():
    """BF16: up to 64 groups of up to 64 values and eight terms, every multiple of eight."""
    for p in (1, 8, 23, 64):
        for q in (1, 9, 40, 64):
            for m1 in (8, 24, 64):
                for m2 in (8, 40, 64):
                    for r in (1, 3, 8):
                        assert native.glu_workspace_size(10, p, q, m1, m2, r, "bf16", True) > 0


def test_binding_rejects():
    S, A, B = torch.ones(2, 3, 4), torch.ones(2, 1, 3, 4), torch.ones(2, 1, 8, 8)
    x = torch.ones(5, 24)
    with pytest.raises(ValueError):
        native.glu_forward(x, S, A, B, dtype="f32")                     # not on a GPU
    with pytest.raises(TypeError):
        native.glu_forward(x, S, A, B, dtype="bf16")
    with pytest.raises(ValueError):
        native.glu_forward(x, S, A, B, activation="relu", dtype="f32")
    with pytest.raises(ValueError):
        native.glu_forward(x, S[0], A, B, dtype="f32")
    with pytest.raises(ValueError):
        native.glu_forward(x, S, A[:, :, :2], B, dtype="f32")
    with pytest.raises(ValueError):
        kfs.KronGLU(96, 96, 32, dtype="tf32")
    with pytest.raises(ValueError):
        kfs.KronGLU(96, 96, 32, activation="relu")
    with pytest.raises(ValueError):
        kfs.KronGLU(96, 100, 32)


def _up(v, n):
    return -(-v // n) * n


def test_documented_limits_of_bf16():
    """Every size within the header's inequalities has a kernel, and the forward does not ask for
    the backward's."""
    pad = lambda m: 16 if m <= 16 else 32 if m <= 32 else _up(m, 64)  # noqa: E731
    takes = {False: 0, True: 0}
    for p in (1, 7, 16, 33, 64, 200, 256, 700, 1024):
        for q in (1, 16, 33, 64, 224, 1024):
            for m1 in (8, 24, 64, 160, 256):
                for m2 in (8, 40, 64, 256):
                    for r in (1, 2, 4, 5, 8, 16, 24):
                        fwd = -(-r // 4) * (_up(p, 16) + pad(m1)) + 2 * pad(m1) <= 646
                        bwd = 2 * -(-r // 8) * (_up(q, 16) + pad(m2)) + 2 * pad(m2) <= 646
                        size = dict(p=p, q=q, m1=m1, m2=m2, r=r)
                        if fwd:       # accepted: with no rows there is nothing to launch
                            assert call(False, N=0, **size) == 0, size
                            takes[False] += 1
                        if fwd and bwd:
                            assert native.glu_workspace_size(8, **size, dtype="bf16",
                                                             backward=True) > 0, size
                            takes[True] += 1
    assert takes[False] > takes[True] > 500


def test_forward_where_the_backward_has_no_kernel():
    """4096 -> 14336, blocks of 64, eight ranks: dX does not fit, the forward does."""
    size = dict(p=64, q=224, m1=64, m2=64, r=8)
    assert call(False, x=None, **size) == 1          # past the sizes, to the pointers
    assert call(False, N=0, **size) == 0
    assert call(True, **size) == 2
    assert "gradients" in native.load().kron_last_error().decode()
    assert native.glu_workspace_size(8, **size, dtype="bf16", backward=True) == 0
    # FP32: a row's tile of the backward has more in it
    size = dict(p=128, q=128, m1=64, m2=64, r=1)
    assert call(False, N=0, dtype=0, **size) == 0
    assert call(True, dtype=0, **size) == 2
    assert native.glu_workspace_size(8, **size, dtype="f32", backward=True) == 0


def test_gated_block_refuses_sizes_that_its_projection_back_lacks():
    """In BF16 the layer has kernels for compiled shapes only: said at construction, not by the
    first forward."""
    for sizes in ((768, 2048, 32, 64, 1), (1024, 1024, 32, 32, 2), (96, 160, 16, 32, 2)):
        *sizes, rank = sizes
        with pytest.raises(ValueError, match="projection back"):
            kfs.KronGatedFFN(*sizes, rank=rank, dtype="bf16")
        kfs.KronGatedFFN(*sizes, rank=rank, dtype="f32")
        kfs.KronGLU(*sizes, rank=rank, dtype="bf16")
    kfs.KronGatedFFN(1024, 1024, 32, rank=4, dtype="bf16")
    kfs.KronGatedFFN(4096, 4096, 64, rank=8, dtype="bf16")
    with pytest.raises(ValueError):
        kfs.KronGatedFFN(768, 2000, 32, 64, dtype="bf16")


def test_binding_rejects_a_workspace_that_is_smaller_than_it_looks():
    """A broadcast buffer has as many elements as a real one and no memory behind them."""
    cpu = torch.device("cpu")
    size = (8, 4, 4, 16, 16, 2)
    n = native.glu_workspace_size(*size, "bf16", True)
    for bad in (torch.empty(1, dtype=torch.uint8).expand(n), torch.empty(2 * n).view(n, 2)[:, 0]):
        with pytest.raises(ValueError, match="contiguous"):
            native._glu_workspace(size, "bf16", True, bad, cpu)
    good = torch.empty(n // 4 + 1)
    _, at, nbytes = native._glu_workspace(size, "bf16", True, good, cpu)
    assert at == good.data_ptr() and nbytes == 4 * good.numel()


def test_binding_rejects_a_stream_of_another_device():
    """The kernels would run on the stream's GPU with pointers of another one."""
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0
    with pytest.raises(ValueError, match="stream"):
        native._on_device(torch.device("cuda", 0), Stream())
