"""ctypes binding of libkronlinear.so (include/kron_linear.h, include/ks_linear.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current CUDA stream.  If the
library has not been built, or a call fails, this module raises -- it never
computes anything itself.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkronlinear.so")

KRON_F32, KRON_TF32, KRON_BF16 = 0, 1, 2
DTYPES = {"f32": KRON_F32, "tf32": KRON_TF32, "bf16": KRON_BF16}
KRON_FLAG_SKIP_ZERO_BLOCKS = 1
KRON_NOALLOC_SCRATCH_BYTES = 8 << 20   # fixed scratch of kron_linear_backward_noalloc

# Paths whose kernels are built into the library.
IMPLEMENTED_PATHS = ("f32", "tf32", "bf16")

STATUS = {0: "KRON_OK", 1: "KRON_ERR_INVALID_ARG", 2: "KRON_ERR_UNSUPPORTED",
          3: "KRON_ERR_ALIGNMENT", 4: "KRON_ERR_WORKSPACE", 5: "KRON_ERR_CUDA",
          6: "KRON_ERR_TIMEOUT"}

# Every symbol include/kron_linear.h declares.
EXPORTS = ("kron_linear_forward", "kron_linear_backward", "kron_linear_backward_l1",
           "kron_linear_backward_noalloc",
           "kron_linear_workspace_size", "kron_vanloan_fit", "kron_vanloan_workspace_size",
           "kron3_linear_forward", "kron3_linear_backward", "kron3_linear_workspace_size",
           "kron_glu_forward", "kron_glu_backward", "kron_glu_workspace_size",
           "kron_distill_forward", "kron_distill_backward", "kron_distill_step",
           "kron_status_string", "kron_last_error", "kron_linear_device_error",
           "kron_linear_abi_version",
           "ks_linear_forward", "ks_linear_backward", "ks_linear_workspace_size")


class KronError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {detail}")


_lib = None


def load(path: str = LIB_PATH):
    """Load the shared library (raises if it is missing: no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing; build it with `python -m kronecker_factored_structured_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i64, I, U, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
    lib.kron_linear_forward.argtypes = [vp, vp, vp, vp, vp, vp, i64, I, I, I, I, I, I, U, vp]
    lib.kron_linear_forward.restype = I
    lib.kron_linear_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                         i64, I, I, I, I, I, I, U, vp, sz, vp]
    lib.kron_linear_backward.restype = I
    lib.kron_linear_backward_l1.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                            i64, I, I, I, I, I, I, U, ctypes.c_double,
                                            vp, sz, vp]
    lib.kron_linear_backward_l1.restype = I
    lib.kron_linear_backward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                 i64, I, I, I, I, I, I, U, vp]
    lib.kron_linear_backward_noalloc.restype = I
    lib.kron_vanloan_workspace_size.argtypes = [I, I, I, I, I]
    lib.kron_vanloan_workspace_size.restype = sz
    lib.kron_vanloan_fit.argtypes = [vp, I, I, I, I, I, vp, I, I, I, vp, vp, vp, vp, vp, sz, vp]
    lib.kron_vanloan_fit.restype = I
    lib.kron3_linear_workspace_size.argtypes = [i64, I, I, I, I, I, I, I, I, I]
    lib.kron3_linear_workspace_size.restype = sz
    lib.kron3_linear_forward.argtypes = [vp, vp, vp, vp, vp, vp, i64, I, I, I, I, I, I, I, I, U,
                                         vp, sz, vp]
    lib.kron3_linear_forward.restype = I
    lib.kron3_linear_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, I, I, I,
                                          I, I, I, I, I, U, vp, sz, vp]
    lib.kron3_linear_backward.restype = I
    D = ctypes.c_double
    lib.kron_glu_workspace_size.argtypes = [i64, I, I, I, I, I, I, I]
    lib.kron_glu_workspace_size.restype = sz
    lib.kron_glu_forward.argtypes = [vp] * 6 + [i64] + [I] * 7 + [U, vp, sz, vp]
    lib.kron_glu_forward.restype = I
    lib.kron_glu_backward.argtypes = [vp] * 11 + [i64] + [I] * 7 + [U, vp, sz, vp]
    lib.kron_glu_backward.restype = I
    lib.kron_distill_forward.argtypes = [vp, i64, vp, vp, I, vp, vp, vp, vp, i64, i64, I, D, D, I,
                                         vp]
    lib.kron_distill_forward.restype = I
    lib.kron_distill_backward.argtypes = [vp, i64, vp, vp, I, vp, vp, vp, vp, vp, i64, i64, i64, I,
                                          D, D, I, vp]
    lib.kron_distill_backward.restype = I
    lib.kron_distill_step.argtypes = [vp, i64, vp, vp, I, vp, vp, vp, vp, i64, i64, i64, I, D, D,
                                      I, vp]
    lib.kron_distill_step.restype = I
    lib.kron_linear_workspace_size.argtypes = [i64, I, I, I, I, I, I]
    lib.kron_linear_workspace_size.restype = sz
    lib.kron_status_string.argtypes = [I]
    lib.kron_status_string.restype = ctypes.c_char_p
    lib.kron_last_error.argtypes = []
    lib.kron_last_error.restype = ctypes.c_char_p
    lib.kron_linear_device_error.argtypes = [I]
    lib.kron_linear_device_error.restype = I
    lib.kron_linear_abi_version.argtypes = []
    lib.kron_linear_abi_version.restype = I
    lib.ks_linear_forward.argtypes = [vp, vp, vp, vp, i64, I, I, I, I, I, U, vp]
    lib.ks_linear_forward.restype = I
    lib.ks_linear_backward.argtypes = [vp, vp, vp, vp, vp, vp, i64, I, I, I, I, I, U, vp, sz, vp]
    lib.ks_linear_backward.restype = I
    lib.ks_linear_workspace_size.argtypes = [i64, I, I, I, I, I]
    lib.ks_linear_workspace_size.restype = sz
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        detail = load().kron_last_error().decode()
        raise KronError(status, detail)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def io_dtype(dtype: str) -> torch.dtype:
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _expect(t, name, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def shapes(S, A, B):
    r, p, q = A.shape
    r2, m1, m2 = B.shape
    if tuple(S.shape) != (p, q) or r2 != r:
        raise ValueError(f"inconsistent factor shapes S{tuple(S.shape)} A{tuple(A.shape)} "
                         f"B{tuple(B.shape)}")
    return p, q, m1, m2, r


def device_error(clear: bool = False) -> None:
    """Raise KronError(KRON_ERR_TIMEOUT) if a kernel's bounded wait gave up."""
    _check(load().kron_linear_device_error(1 if clear else 0))


def workspace_size(N, p, q, m1, m2, r, dtype="tf32") -> int:
    return int(load().kron_linear_workspace_size(N, p, q, m1, m2, r, DTYPES[dtype]))


def forward(x, S, A, B, bias=None, dtype="tf32", flags=0, out=None, stream=None):
    """y = x W + bias with W = sum_i kron(S*A_i, B_i), on the library's kernels."""
    p, q, m1, m2, r = shapes(S, A, B)
    N = x.shape[0]
    t = io_dtype(dtype)
    _expect(x, "x", t, (N, p * m1))
    for name, v, shp in (("S", S, (p, q)), ("A", A, (r, p, q)), ("B", B, (r, m1, m2))):
        _expect(v, name, t, shp)
    if bias is not None:
        _expect(bias, "bias", t, (q * m2,))
    if out is None:
        out = torch.empty(N, q * m2, dtype=t, device=x.device)
    _expect(out, "y", t, (N, q * m2))
    _check(load().kron_linear_forward(_ptr(x), _ptr(S), _ptr(A), _ptr(B), _ptr(bias), _ptr(out),
                                      N, p, q, m1, m2, r, DTYPES[dtype], flags, _stream(stream)))
    return out


def backward(x, S, A, B, dY, dtype="tf32", flags=0, need_dx=True, need_dbias=True,
             workspace=None, grads=None, stream=None, l1=0.0):
    """Gradients of <dY, y>: returns dict(dX, dS, dA, dB, dbias).

    dX has the I/O dtype; dS, dA, dB and dbias are float32.  ``grads`` may hold
    preallocated outputs (same keys); ``workspace`` a preallocated uint8 buffer.
    ``l1`` > 0 adds the gradient l1 * sign(S) of the penalty l1 * sum|S| to dS inside the
    library's dS epilogue (kron_linear_backward_l1).
    """
    p, q, m1, m2, r = shapes(S, A, B)
    N = x.shape[0]
    t = io_dtype(dtype)
    _expect(x, "x", t, (N, p * m1))
    _expect(dY, "dY", t, (N, q * m2))
    for name, v, shp in (("S", S, (p, q)), ("A", A, (r, p, q)), ("B", B, (r, m1, m2))):
        _expect(v, name, t, shp)
    dev = x.device
    g = dict(grads or {})
    f32 = torch.float32
    if need_dx and g.get("dX") is None:
        g["dX"] = torch.empty(N, p * m1, dtype=t, device=dev)
    if not need_dx:
        g["dX"] = None
    for k, shp in (("dS", (p, q)), ("dA", (r, p, q)), ("dB", (r, m1, m2))):
        if g.get(k) is None:
            g[k] = torch.empty(shp, dtype=f32, device=dev)
        _expect(g[k], k, f32, shp)
    if need_dbias and g.get("dbias") is None:
        g["dbias"] = torch.empty(q * m2, dtype=f32, device=dev)
    if not need_dbias:
        g["dbias"] = None
    ws_bytes = workspace_size(N, p, q, m1, m2, r, dtype)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    ptrs = (_ptr(x), _ptr(S), _ptr(A), _ptr(B), _ptr(dY), _ptr(g["dX"]), _ptr(g["dS"]),
            _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dbias"]), N, p, q, m1, m2, r, DTYPES[dtype],
            flags)
    tail = (_ptr(workspace), workspace.numel(), _stream(stream))
    if l1:
        _check(load().kron_linear_backward_l1(*ptrs, float(l1), *tail))
    else:
        _check(load().kron_linear_backward(*ptrs, *tail))
    return g


def vanloan_fit(W, p, q, m1, m2, r, k=None, power_iters=2, normalize=True, omega=None,
                seed=0, stream=None):
    """Rank-r Kronecker fit of a dense float32 CUDA matrix W ((p*m1) x (q*m2)) by the
    library's kron_vanloan_fit; returns dict(S = ones, A [r][p][q], B [r][m1][m2],
    sigma [k], alpha).  ``omega`` ([k][m1*m2] float32) is the random test matrix; by default
    it is drawn here with torch (seeded), k = r + 8 capped by the sizes."""
    if k is None:
        k = min(r + 8, 64, p * q, m1 * m2)
    _expect(W, "W", torch.float32, (p * m1, q * m2))
    dev = W.device
    if omega is None:
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        omega = torch.randn(k, m1 * m2, device=dev, generator=g)
    _expect(omega, "omega", torch.float32, (k, m1 * m2))
    A = torch.empty(r, p, q, device=dev)
    B = torch.empty(r, m1, m2, device=dev)
    sigma = torch.empty(k, device=dev)
    alpha = torch.empty(4, device=dev)
    lib = load()
    wsb = int(lib.kron_vanloan_workspace_size(p, q, m1, m2, k))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    _check(lib.kron_vanloan_fit(_ptr(W), p, q, m1, m2, r, _ptr(omega), k, power_iters,
                                1 if normalize else 0, _ptr(A), _ptr(B), _ptr(sigma), _ptr(alpha),
                                _ptr(ws), ws.numel(), _stream(stream)))
    return {"S": torch.ones(p, q, device=dev), "A": A, "B": B, "sigma": sigma,
            "alpha": alpha[:1]}


def _shapes3(A, B, C):
    r, p, q = A.shape
    r2, m1, m2 = B.shape
    r3, s1, s2 = C.shape
    if r2 != r or r3 != r:
        raise ValueError("A, B and C must hold the same number of terms")
    return p, q, m1, m2, s1, s2, r


def forward3(x, A, B, C, bias=None, dtype="tf32", flags=0, stream=None):
    """Triple Kronecker layer y = x W + bias, W = sum_i kron(A_i, kron(B_i, C_i))."""
    p, q, m1, m2, s1, s2, r = _shapes3(A, B, C)
    N = x.shape[0]
    t = io_dtype(dtype)
    _expect(x, "x", t, (N, p * m1 * s1))
    for name, v, shp in (("A", A, (r, p, q)), ("B", B, (r, m1, m2)), ("C", C, (r, s1, s2))):
        _expect(v, name, t, shp)
    y = torch.empty(N, q * m2 * s2, dtype=t, device=x.device)
    lib = load()
    n = int(lib.kron3_linear_workspace_size(N, p, q, m1, m2, s1, s2, r, DTYPES[dtype], 0))
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=x.device)
    _check(lib.kron3_linear_forward(_ptr(x), _ptr(A), _ptr(B), _ptr(C), _ptr(bias), _ptr(y), N, p,
                                    q, m1, m2, s1, s2, r, DTYPES[dtype], flags, _ptr(ws),
                                    ws.numel(), _stream(stream)))
    return y


def backward3(x, A, B, C, dY, dtype="tf32", flags=0, stream=None):
    """Gradients of <dY, y> for the triple layer: dict(dX, dA, dB, dC, dbias)."""
    p, q, m1, m2, s1, s2, r = _shapes3(A, B, C)
    N = x.shape[0]
    t = io_dtype(dtype)
    _expect(x, "x", t, (N, p * m1 * s1))
    _expect(dY, "dY", t, (N, q * m2 * s2))
    dev = x.device
    g = {"dX": torch.empty(N, p * m1 * s1, dtype=t, device=dev),
         "dA": torch.empty(r, p, q, device=dev), "dB": torch.empty(r, m1, m2, device=dev),
         "dC": torch.empty(r, s1, s2, device=dev), "dbias": torch.empty(q * m2 * s2, device=dev)}
    lib = load()
    n = int(lib.kron3_linear_workspace_size(N, p, q, m1, m2, s1, s2, r, DTYPES[dtype], 1))
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    _check(lib.kron3_linear_backward(_ptr(x), _ptr(A), _ptr(B), _ptr(C), _ptr(dY), _ptr(g["dX"]),
                                     _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dbias"]),
                                     N, p, q, m1, m2, s1, s2, r, DTYPES[dtype], flags, _ptr(ws),
                                     ws.numel(), _stream(stream)))
    return g


# ---- Kronecker-sparse factor (include/ks_linear.h) ----

def ks_pattern(w):
    """(a, b, c, d) of the values w, laid out [a][d][b][c]."""
    if w.dim() != 4:
        raise ValueError(f"w must have shape (a, d, b, c), got {tuple(w.shape)}")
    a, d, b, c = w.shape
    return a, b, c, d


def ks_workspace_size(N, a, b, c, d) -> int:
    return int(load().ks_linear_workspace_size(N, a, b, c, d, KRON_F32))


def ks_forward(x, w, bias=None, out=None, stream=None):
    """y = x K + bias for the KS matrix K of pattern (a, b, c, d) with values w."""
    a, b, c, d = ks_pattern(w)
    N = x.shape[0]
    f32 = torch.float32
    _expect(x, "x", f32, (N, a * b * d))
    _expect(w, "w", f32, (a, d, b, c))
    if bias is not None:
        _expect(bias, "bias", f32, (a * c * d,))
    if out is None:
        out = torch.empty(N, a * c * d, dtype=f32, device=x.device)
    _expect(out, "y", f32, (N, a * c * d))
    _check(load().ks_linear_forward(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), N, a, b, c, d,
                                    KRON_F32, 0, _stream(stream)))
    return out


def ks_backward(x, w, dY, need_dx=True, need_dbias=True, workspace=None, grads=None,
                stream=None):
    """Gradients of <dY, y> for the KS factor: dict(dX, dw, dbias) (None where not asked)."""
    a, b, c, d = ks_pattern(w)
    N = x.shape[0]
    f32 = torch.float32
    _expect(x, "x", f32, (N, a * b * d))
    _expect(w, "w", f32, (a, d, b, c))
    _expect(dY, "dY", f32, (N, a * c * d))
    dev = x.device
    g = dict(grads or {})
    if need_dx and g.get("dX") is None:
        g["dX"] = torch.empty(N, a * b * d, dtype=f32, device=dev)
    if not need_dx:
        g["dX"] = None
    if g.get("dw") is None:
        g["dw"] = torch.empty(a, d, b, c, dtype=f32, device=dev)
    _expect(g["dw"], "dw", f32, (a, d, b, c))
    if need_dbias and g.get("dbias") is None:
        g["dbias"] = torch.empty(a * c * d, dtype=f32, device=dev)
    if not need_dbias:
        g["dbias"] = None
    if workspace is None:
        workspace = torch.empty(ks_workspace_size(N, a, b, c, d), dtype=torch.uint8, device=dev)
    _check(load().ks_linear_backward(_ptr(x), _ptr(w), _ptr(dY), _ptr(g["dX"]), _ptr(g["dw"]),
                                     _ptr(g["dbias"]), N, a, b, c, d, KRON_F32, 0,
                                     _ptr(workspace), workspace.numel(), _stream(stream)))
    return g


# Checks and launch helpers of the calls below.  A short call spends more time here than on the
# GPU, so a tensor that is as it should be passes in one comparison.

def _need(t, name, dtype, shape, dev):
    """t is a contiguous CUDA tensor of this dtype and shape on device dev."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev.index
            and t.is_contiguous()):
        return
    _expect(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, not on {dev}")


def _on_device(dev, stream):
    """Context in which dev is the current device, and memory that is allocated belongs to the
    stream that the call runs on (a workspace may be handed out again once it returns)."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
        return torch.cuda.stream(stream)
    return _NOTHING if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


_NOTHING = contextlib.nullcontext()


def _raw_stream(stream, dev):
    return (torch._C._cuda_getCurrentRawStream(dev.index) if stream is None
            else stream.cuda_stream)


def _at(t):
    return None if t is None else t.data_ptr()


# ---- gated half of a feed-forward block: h = act(x Wg + bg) * (x Wu + bu) ----

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "sigmoid": 3}


def glu_shapes(S, A, B):
    """(p, q, m1, m2, r) of factors stacked [gate, up]."""
    if S.dim() != 3 or A.dim() != 4 or B.dim() != 4:
        raise ValueError("S must have shape (2, p, q), A (2, r, p, q) and B (2, r, m1, m2)")
    two, r, p, q = A.shape
    m1, m2 = B.shape[2:]
    if two != 2 or tuple(S.shape) != (2, p, q) or tuple(B.shape[:2]) != (2, r):
        raise ValueError(f"inconsistent factor shapes S{tuple(S.shape)} A{tuple(A.shape)} "
                         f"B{tuple(B.shape)}")
    return p, q, m1, m2, r


def _glu_args(x, S, A, B, bias, activation, dtype):
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    p, q, m1, m2, r = glu_shapes(S, A, B)
    if x.dim() != 2:
        raise ValueError(f"x must have shape (N, {p * m1}), got {tuple(x.shape)}")
    N = x.shape[0]
    t, dev = io_dtype(dtype), x.device
    _need(x, "x", t, (N, p * m1), dev)
    _need(S, "S", t, (2, p, q), dev)
    _need(A, "A", t, (2, r, p, q), dev)
    _need(B, "B", t, (2, r, m1, m2), dev)
    if bias is not None:
        _need(bias, "bias", t, (2, q * m2), dev)
    return (N, p, q, m1, m2, r), t, dev


def glu_workspace_size(N, p, q, m1, m2, r, dtype="bf16", backward=False) -> int:
    return int(load().kron_glu_workspace_size(N, p, q, m1, m2, r, DTYPES[dtype],
                                              1 if backward else 0))


def _glu_workspace(sizes, dtype, backward, workspace, dev):
    """(workspace tensor to keep alive, address, bytes)"""
    if workspace is None:
        # the BF16 forward needs none
        n = glu_workspace_size(*sizes, dtype, backward) if backward or dtype != "bf16" else 0
        if not n:
            return None, None, 0
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    elif workspace.device != dev:
        raise ValueError(f"workspace is on {workspace.device}, not on {dev}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def glu_forward(x, S, A, B, bias=None, activation="silu", dtype="bf16", out=None, workspace=None,
                stream=None):
    """h = act(x Wg + bg) * (x Wu + bu), W* = sum_i kron(S* (.) A*_i, B*_i); S [2][p][q],
    A [2][r][p][q], B [2][r][m1][m2] and bias [2][q*m2] hold the gate, then the up projection.
    dtype "f32" or "bf16"."""
    sizes, t, dev = _glu_args(x, S, A, B, bias, activation, dtype)
    shape = (sizes[0], sizes[2] * sizes[4])
    with _on_device(dev, stream):
        if out is None:
            out = x.new_empty(shape)
        else:
            _need(out, "h", t, shape, dev)
        keep, ws, ws_bytes = _glu_workspace(sizes, dtype, False, workspace, dev)
        _check(load().kron_glu_forward(x.data_ptr(), S.data_ptr(), A.data_ptr(), B.data_ptr(),
                                       _at(bias), out.data_ptr(), *sizes, ACTIVATIONS[activation],
                                       DTYPES[dtype], 0, ws, ws_bytes, _raw_stream(stream, dev)))
    return out


def glu_backward(x, S, A, B, dH, bias=None, activation="silu", dtype="bf16", need_dx=True,
                 need_dbias=True, workspace=None, grads=None, stream=None):
    """Gradients of <dH, h>: dict(dX, dS, dA, dB, dbias) in the tensors' own dtype (None where
    not asked).  ``grads`` may hold preallocated outputs."""
    sizes, t, dev = _glu_args(x, S, A, B, bias, activation, dtype)
    N, p, q, m1, m2, r = sizes
    _need(dH, "dH", t, (N, q * m2), dev)
    g = dict(grads or {})
    with _on_device(dev, stream):
        for k, shp, need in (("dX", (N, p * m1), need_dx), ("dS", (2, p, q), True),
                             ("dA", (2, r, p, q), True), ("dB", (2, r, m1, m2), True),
                             ("dbias", (2, q * m2), need_dbias)):
            if not need:
                g[k] = None
            elif g.get(k) is None:
                g[k] = x.new_empty(shp)
            else:
                _need(g[k], k, t, shp, dev)
        keep, ws, ws_bytes = _glu_workspace(sizes, dtype, True, workspace, dev)
        _check(load().kron_glu_backward(x.data_ptr(), S.data_ptr(), A.data_ptr(), B.data_ptr(),
                                        _at(bias), dH.data_ptr(), _at(g["dX"]), _at(g["dS"]),
                                        _at(g["dA"]), _at(g["dB"]), _at(g["dbias"]), *sizes,
                                        ACTIVATIONS[activation], DTYPES[dtype], 0, ws, ws_bytes,
                                        _raw_stream(stream, dev)))
    return g


# ---- distillation loss against a teacher's top logits ----

def _rows(t, name, dtype, N, V):
    """Row stride of a matrix whose rows are contiguous and may lie further apart than their
    length."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (N, V):
        raise ValueError(f"{name} must have shape {(N, V)}, got {tuple(t.shape)}")
    ld, one = t.stride()
    if not t.is_cuda or (V > 1 and one != 1) or (N > 1 and ld < V):
        raise ValueError(f"{name} must be a CUDA matrix with contiguous rows")
    return ld if N > 1 else V


def _distill_args(logits, values, indices, labels, weights, label_weight):
    if logits.dim() != 2 or values.dim() != 2:
        raise ValueError("logits must have shape (N, V), values and indices (N, K)")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    N, V = logits.shape
    K = values.shape[1]
    dev = logits.device
    ld = _rows(logits, "logits", logits.dtype, N, V)
    _need(values, "values", torch.float32, (N, K), dev)
    if indices.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"indices must be int32 or int64, got {indices.dtype}")
    _need(indices, "indices", indices.dtype, (N, K), dev)
    if label_weight and labels is None:
        raise ValueError("labels are needed when label_weight is above 0")
    if labels is not None:
        _need(labels, "labels", torch.int64, (N,), dev)
    if weights is not None:
        _need(weights, "weights", torch.float32, (N,), dev)
    head = (logits.data_ptr(), ld, values.data_ptr(), indices.data_ptr(),
            8 if indices.dtype is torch.int64 else 4, _at(labels), _at(weights))
    return N, V, K, head, KRON_BF16 if logits.dtype is torch.bfloat16 else KRON_F32, dev


def _dlogits(logits, out):
    N, V = logits.shape
    if out is None:
        return logits.new_empty((N, V)), V
    ld = _rows(out, "dlogits", logits.dtype, N, V)
    if out.device != logits.device:
        raise ValueError(f"dlogits is on {out.device}, not on {logits.device}")
    return out, ld


def distill_forward(logits, values, indices, labels=None, weights=None, temperature=1.0,
                    label_weight=0.0, stream=None):
    """Loss of each row against the teacher's top logits: dict(loss [N], lse [N][2])."""
    N, V, K, head, dtype, dev = _distill_args(logits, values, indices, labels, weights,
                                              label_weight)
    with _on_device(dev, stream):
        loss = values.new_empty(N)
        lse = values.new_empty((N, 2))
        _check(load().kron_distill_forward(*head, loss.data_ptr(), lse.data_ptr(), N, V, K,
                                           temperature, label_weight, dtype,
                                           _raw_stream(stream, dev)))
    return {"loss": loss, "lse": lse}


def distill_backward(logits, values, indices, lse, dloss=None, labels=None, weights=None,
                     temperature=1.0, label_weight=0.0, out=None, stream=None):
    """Gradient of <dloss, loss> in the logits (``dloss`` None: ones).  ``out`` may be the
    logits themselves, which the gradient then overwrites."""
    N, V, K, head, dtype, dev = _distill_args(logits, values, indices, labels, weights,
                                              label_weight)
    _need(lse, "lse", torch.float32, (N, 2), dev)
    if dloss is not None:
        _need(dloss, "dloss", torch.float32, (N,), dev)
    with _on_device(dev, stream):
        out, ld_out = _dlogits(logits, out)
        _check(load().kron_distill_backward(*head, lse.data_ptr(), _at(dloss), out.data_ptr(),
                                            ld_out, N, V, K, temperature, label_weight, dtype,
                                            _raw_stream(stream, dev)))
    return out


def distill_step(logits, values, indices, labels=None, weights=None, temperature=1.0,
                 label_weight=0.0, out=None, stream=None):
    """Loss of each row and the gradient of their sum in one call: dict(loss [N], dlogits).
    ``out`` may be the logits themselves.  Where the logits' rows lie further apart than their
    length, an ``out`` of the same stride is stored fastest."""
    N, V, K, head, dtype, dev = _distill_args(logits, values, indices, labels, weights,
                                              label_weight)
    with _on_device(dev, stream):
        loss = values.new_empty(N)
        out, ld_out = _dlogits(logits, out)
        _check(load().kron_distill_step(*head, loss.data_ptr(), out.data_ptr(), ld_out, N, V, K,
                                        temperature, label_weight, dtype,
                                        _raw_stream(stream, dev)))
    return {"loss": loss, "dlogits": out}
