"""Refusals of the distillation loss: every call below fails a host-side check, so nothing is
launched and no GPU is needed."""
import ctypes

import pytest
import torch

import kronecker_factored_structured_b200 as kfs
from kronecker_factored_structured_b200 import native

V_ = ctypes.c_void_p
OK = V_(0x10000)           # never dereferenced
ODD = V_(0x10001)


def call(entry, logits=OK, ld=100, values=OK, indices=OK, index_bytes=8, labels=OK, weights=None,
         loss=OK, lse=OK, dlogits=V_(0x20000), ld_out=100, N=4, V=100, K=5, tau=2.0, lam=0.5,
         dtype=0):
    lib = native.load()
    head = (logits, ld, values, indices, index_bytes, labels, weights)
    tail = (N, V, K, tau, lam, dtype, None)
    if entry == "forward":
        return lib.kron_distill_forward(*head, loss, lse, *tail)
    if entry == "backward":
        return lib.kron_distill_backward(*head, lse, None, dlogits, ld_out, *tail)
    return lib.kron_distill_step(*head, loss, dlogits, ld_out, *tail)


COMMON = [(dict(dtype=1), 2), (dict(dtype=9), 2), (dict(N=-1), 1), (dict(N=1 << 31), 1),
          (dict(V=0), 1), (dict(V=(1 << 30) + 1, ld=1 << 31, ld_out=1 << 31), 1),
          (dict(K=0), 1), (dict(K=1025), 2), (dict(ld=99), 1), (dict(index_bytes=2), 1),
          (dict(tau=0.0), 1), (dict(tau=-1.0), 1), (dict(tau=float("nan")), 1),
          (dict(tau=2e3), 1), (dict(tau=0.01), 1), (dict(lam=-0.1), 1), (dict(lam=1.5), 1),
          (dict(lam=float("nan")), 1), (dict(labels=None), 1), (dict(logits=None), 1),
          (dict(values=None), 1), (dict(indices=None), 1), (dict(logits=ODD), 3),
          (dict(logits=V_(0x10002)), 3), (dict(logits=ODD, dtype=2), 3), (dict(values=ODD), 3),
          (dict(indices=V_(0x10004)), 3), (dict(weights=ODD), 3), (dict(labels=ODD), 3)]


@pytest.mark.parametrize("entry", ["forward", "backward", "step"])
@pytest.mark.parametrize("kwargs,status", COMMON)
def test_rejects(entry, kwargs, status):
    assert call(entry, **kwargs) == status
    assert native.load().kron_last_error().decode() != ""


@pytest.mark.parametrize("entry,kwargs,status", [
    ("forward", dict(loss=None), 1), ("forward", dict(loss=ODD), 3), ("forward", dict(lse=ODD), 3),
    ("backward", dict(lse=None), 1), ("backward", dict(dlogits=None), 1),
    ("backward", dict(ld_out=99), 1), ("backward", dict(dlogits=ODD), 3),
    ("step", dict(loss=None), 1), ("step", dict(dlogits=None), 1), ("step", dict(ld_out=50), 1),
    ("step", dict(dlogits=V_(0x20002)), 3),
    ("step", dict(dlogits=OK, ld=128, ld_out=100), 1),       # in place with another stride
    ("backward", dict(dlogits=OK, ld=128, ld_out=100), 1),
])
def test_rejects_outputs(entry, kwargs, status):
    assert call(entry, **kwargs) == status


def test_no_rows_is_fine():
    for entry in ("forward", "backward", "step"):
        assert call(entry, N=0, logits=None, values=None, indices=None, labels=None, loss=None,
                    lse=None, dlogits=None, weights=None) == 0
        assert native.load().kron_last_error().decode() == ""


def test_binding_rejects():
    x, v, i = torch.zeros(3, 10), torch.zeros(3, 2), torch.zeros(3, 2, dtype=torch.int64)
    with pytest.raises(ValueError):
        native.distill_forward(x, v, i)                       # not on a GPU
    with pytest.raises(TypeError):
        native.distill_forward(x.half(), v, i)
    with pytest.raises(ValueError):
        native.distill_forward(x[0], v, i)
    with pytest.raises(ValueError):
        kfs.distill_loss(x, v, i, reduction="max")
