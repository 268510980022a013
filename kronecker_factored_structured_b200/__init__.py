"""B200-native sum-of-Kronecker-products linear layer.

    y = x W + bias,   W = sum_{i<r} kron(S (.) A_i, B_i)

(page "kronecker-layer-benchmark", section "1. Build W, then multiply") computed
with the vec trick by the hand-written sm_100a kernels of libkronlinear.so; W is
never materialised.  ``native`` is the ctypes binding of the C ABI
(include/kron_linear.h); ``KronLinearFunction`` / ``KronLinear`` wrap it for
autograd.  PyTorch is used for device memory and streams only.

The same library holds the Kronecker-sparse factor of the page "Fast Inference
with Kronecker-Sparse Matrices" (support kron(I_a, kron(1_{b x c}, I_d)),
include/ks_linear.h): ``native.ks_forward`` / ``native.ks_backward``, wrapped by
``KSLinearFunction`` / ``KSLinear``.

``KronGLU`` is the gated half of a feed-forward block, act(x Wg + bg) * (x Wu + bu), over two
projections of the layer's form; ``KronGatedFFN`` puts a ``KronLinear`` behind it.

``distill_loss`` / ``DistillLoss`` train a compressed model on its dense original's top logits
(``native.distill_forward`` / ``distill_backward``; ``native.distill_step`` gives the loss and
its gradient from one call).
"""
from __future__ import annotations

import math

import torch

from . import accounting, native
from .native import KronError, backward, forward, workspace_size

__all__ = ["native", "accounting", "forward", "backward", "workspace_size", "KronError",
           "KronLinearFunction", "KronLinear", "kron_linear", "KSLinearFunction", "KSLinear",
           "ks_linear", "KronGLUFunction", "KronGLU", "kron_glu", "KronGatedFFN",
           "DistillFunction", "DistillLoss", "distill_loss"]


class KronLinearFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run in the CUDA library.

    Nothing but the inputs is saved; the backward recomputes X_n B_i on chip.
    Factor gradients come back in float32 and are cast to the parameters' dtype.
    ``l1`` > 0 makes S's gradient include that of the penalty l1 * sum|S| (added in the
    library's dS epilogue); the penalty's value is not part of the output.
    """

    @staticmethod
    def forward(ctx, x, S, A, B, bias, dtype, flags, l1=0.0):
        ctx.save_for_backward(x, S, A, B)
        ctx.dtype, ctx.flags, ctx.has_bias, ctx.l1 = dtype, flags, bias is not None, l1
        return forward(x, S, A, B, bias, dtype=dtype, flags=flags)

    @staticmethod
    def backward(ctx, dY):
        x, S, A, B = ctx.saved_tensors
        g = backward(x, S, A, B, dY.contiguous(), dtype=ctx.dtype, flags=ctx.flags,
                     need_dx=ctx.needs_input_grad[0], need_dbias=ctx.has_bias, l1=ctx.l1)
        cast = lambda t, like: None if t is None else t.to(like.dtype)
        dbias = cast(g["dbias"], S) if ctx.has_bias else None
        return (g["dX"], cast(g["dS"], S), cast(g["dA"], A), cast(g["dB"], B), dbias,
                None, None, None)


def kron_linear(x, S, A, B, bias=None, dtype="tf32", flags=0, l1=0.0):
    return KronLinearFunction.apply(x, S, A, B, bias, dtype, flags, l1)


class KronLinear(torch.nn.Module):
    """Drop-in linear layer with W = sum_i kron(S (.) A_i, B_i), W of shape
    (p*m1) x (q*m2); initialised as on the page "kronecker-layer-benchmark"
    (S = ones, A_i ~ randn/sqrt(p), B_i ~ randn/sqrt(m1), bias = zeros).

    ``l1`` > 0 trains S under the page's penalty l1 * sum|S| with its gradient fused into
    the backward's dS epilogue; the loss the caller computes then leaves the penalty out."""

    def __init__(self, in_features, out_features, block_in, block_out=None, rank=1,
                 bias=True, dtype="tf32", flags=0, device=None, l1=0.0):
        super().__init__()
        block_out = block_in if block_out is None else block_out
        if in_features % block_in or out_features % block_out:
            raise ValueError("features must be multiples of the block size")
        p, q = in_features // block_in, out_features // block_out
        t = native.io_dtype(dtype)
        kw = dict(device=device, dtype=t)
        self.S = torch.nn.Parameter(torch.ones(p, q, **kw))
        self.A = torch.nn.Parameter(torch.randn(rank, p, q, **kw) / math.sqrt(p))
        self.B = torch.nn.Parameter(torch.randn(rank, block_in, block_out, **kw) / math.sqrt(block_in))
        self.bias = torch.nn.Parameter(torch.zeros(out_features, **kw)) if bias else None
        self.path, self.flags, self.l1 = dtype, flags, float(l1)

    def forward(self, x):
        shp = x.shape
        y = kron_linear(x.reshape(-1, shp[-1]).contiguous(), self.S, self.A, self.B, self.bias,
                        self.path, self.flags, self.l1)
        return y.reshape(*shp[:-1], y.shape[-1])


class KSLinearFunction(torch.autograd.Function):
    """Autograd wrapper of the Kronecker-sparse factor; both passes run in the CUDA library."""

    @staticmethod
    def forward(ctx, x, w, bias):
        ctx.save_for_backward(x, w)
        ctx.has_bias = bias is not None
        return native.ks_forward(x, w, bias)

    @staticmethod
    def backward(ctx, dY):
        x, w = ctx.saved_tensors
        g = native.ks_backward(x, w, dY.contiguous(), need_dx=ctx.needs_input_grad[0],
                               need_dbias=ctx.has_bias)
        return g["dX"], g["dw"], g["dbias"]


def ks_linear(x, w, bias=None):
    return KSLinearFunction.apply(x, w, bias)


class KSLinear(torch.nn.Module):
    """Linear layer y = x K + bias whose weight K is Kronecker-sparse with pattern
    (a, b, c, d): supp K = kron(I_a, kron(1_{b x c}, I_d)), in = a*b*d, out = a*c*d.
    The a*d dense b x c blocks are initialised with std 1/sqrt(b) (each output sums b
    inputs); FP32 only.  Butterfly and Monarch layers are sequences of these."""

    def __init__(self, a, b, c, d, bias=True, device=None):
        super().__init__()
        kw = dict(device=device, dtype=torch.float32)
        self.pattern = (a, b, c, d)
        self.w = torch.nn.Parameter(torch.randn(a, d, b, c, **kw) / math.sqrt(b))
        self.bias = torch.nn.Parameter(torch.zeros(a * c * d, **kw)) if bias else None

    def forward(self, x):
        shp = x.shape
        y = ks_linear(x.reshape(-1, shp[-1]).contiguous(), self.w, self.bias)
        return y.reshape(*shp[:-1], y.shape[-1])


class KronGLUFunction(torch.autograd.Function):
    """Autograd wrapper of the gated half; both passes run in the CUDA library, and the
    backward forms the pre-activations again from the saved inputs."""

    @staticmethod
    def forward(ctx, x, S, A, B, bias, activation, dtype):
        ctx.save_for_backward(x, S, A, B, bias)
        ctx.activation, ctx.dtype = activation, dtype
        return native.glu_forward(x, S, A, B, bias, activation, dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dH):
        x, S, A, B, bias = ctx.saved_tensors
        g = native.glu_backward(x, S, A, B, dH.contiguous(), bias, ctx.activation, ctx.dtype,
                                need_dx=ctx.needs_input_grad[0], need_dbias=bias is not None)
        return g["dX"], g["dS"], g["dA"], g["dB"], g["dbias"], None, None


def kron_glu(x, S, A, B, bias=None, activation="silu", dtype="bf16"):
    """act(x Wg + bg) * (x Wu + bu) with W* = sum_i kron(S* (.) A*_i, B*_i): S (2, p, q),
    A (2, r, p, q), B (2, r, m1, m2) and bias (2, q*m2) hold the gate, then the up projection."""
    return KronGLUFunction.apply(x, S, A, B, bias, activation, dtype)


class KronGLU(torch.nn.Module):
    """Gated half of a feed-forward block: two Kronecker-factored projections, an activation
    ("silu", "gelu", "gelu_tanh", "sigmoid") and the product.  Factors are initialised as
    ``KronLinear``'s.  dtype "bf16" (tensor cores) or "f32" (exact)."""

    def __init__(self, in_features, hidden_features, block_in, block_out=None, rank=1, bias=True,
                 activation="silu", dtype="bf16", device=None):
        super().__init__()
        block_out = block_in if block_out is None else block_out
        if in_features % block_in or hidden_features % block_out:
            raise ValueError("features must be multiples of the block size")
        if dtype not in ("f32", "bf16"):
            raise ValueError(f"the gated half runs on 'f32' and 'bf16', got {dtype!r}")
        if activation not in native.ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(native.ACTIVATIONS)}, "
                             f"got {activation!r}")
        p, q = in_features // block_in, hidden_features // block_out
        kw = dict(device=device, dtype=native.io_dtype(dtype))
        self.S = torch.nn.Parameter(torch.ones(2, p, q, **kw))
        self.A = torch.nn.Parameter(torch.randn(2, rank, p, q, **kw) / math.sqrt(p))
        self.B = torch.nn.Parameter(torch.randn(2, rank, block_in, block_out, **kw)
                                    / math.sqrt(block_in))
        self.bias = (torch.nn.Parameter(torch.zeros(2, hidden_features, **kw)) if bias else None)
        self.activation, self.path = activation, dtype

    def forward(self, x):
        h = kron_glu(x.reshape(-1, x.shape[-1]).contiguous(), self.S, self.A, self.B, self.bias,
                     self.activation, self.path)
        return h.reshape(*x.shape[:-1], h.shape[-1])


class KronGatedFFN(torch.nn.Module):
    """Gated feed-forward block of Kronecker-factored projections: ``KronGLU`` (``glu``) to the
    hidden width, ``KronLinear`` (``down``) back, whose shapes and dtypes are its own.  "f32" takes
    run-time sizes; in "bf16" ``down`` has kernels for the layer's compiled shapes only, and other
    sizes are refused here (ValueError): put a ``KronGLU`` before a projection of your own."""

    def __init__(self, features, hidden_features, block, hidden_block=None, rank=1, bias=True,
                 activation="silu", dtype="bf16", device=None):
        super().__init__()
        hidden_block = block if hidden_block is None else hidden_block
        if dtype == "bf16" and not (features % block or hidden_features % hidden_block):
            down = (hidden_features // hidden_block, features // block, hidden_block, block, rank)
            if not native.workspace_size(1, *down, dtype):
                raise ValueError(
                    "no bf16 kernel for the projection back: p=%d q=%d m1=%d m2=%d r=%d is not one "
                    "of the layer's compiled shapes (dtype='f32' takes run-time sizes)" % down)
        self.glu = KronGLU(features, hidden_features, block, hidden_block, rank, bias, activation,
                           dtype, device)
        self.down = KronLinear(hidden_features, features, hidden_block, block, rank, bias, dtype,
                               device=device)

    def forward(self, x):
        return self.down(self.glu(x))


class DistillFunction(torch.autograd.Function):
    """Autograd wrapper of the distillation loss: a loss per row, the gradients in the logits and,
    where they need one, in the rows' weights."""

    @staticmethod
    def forward(ctx, logits, values, indices, labels, weights, temperature, label_weight):
        g = native.distill_forward(logits, values, indices, labels, weights, temperature,
                                   label_weight)
        ctx.save_for_backward(logits, values, indices, labels, weights, g["lse"])
        ctx.temperature, ctx.label_weight = temperature, label_weight
        return g["loss"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        logits, values, indices, labels, weights, lse = ctx.saved_tensors
        dloss = dloss.contiguous()
        d = dw = None
        if ctx.needs_input_grad[0]:
            d = native.distill_backward(logits, values, indices, lse, dloss, labels, weights,
                                        ctx.temperature, ctx.label_weight)
        if ctx.needs_input_grad[4]:
            # the row's loss without its weight, which the weighted one does not give at zero
            dw = dloss * native.distill_forward(logits, values, indices, labels, None,
                                                ctx.temperature, ctx.label_weight)["loss"]
        return d, None, None, None, dw, None, None


def distill_loss(logits, values, indices, labels=None, weights=None, temperature=1.0,
                 label_weight=0.0, reduction="mean"):
    """(1 - label_weight) temperature^2 KL(teacher || student) over the teacher's top logits
    plus label_weight times the cross-entropy with ``labels``, per row of ``logits``.

    ``values`` (float32) and ``indices`` hold the teacher's logits of each row and their
    columns, an index outside the vocabulary being no entry; shapes are (..., V), (..., K) and
    (...), of any strides (logits whose rows are not contiguous are copied).  ``weights``
    multiplies the rows.  reduction: "none" (the rows' losses), "sum", or "mean" (the sum over the
    sum of ``weights``, or over the rows without them).  ``logits`` and ``weights`` are
    differentiable (the backward forms the rows' losses again for the weights); the teacher gets
    no gradient.
    """
    if reduction not in ("none", "sum", "mean"):
        raise ValueError(f"reduction must be 'none', 'sum' or 'mean', got {reduction!r}")
    lead = logits.shape[:-1]
    flat = lambda t: None if t is None else t.reshape(-1).contiguous()  # noqa: E731
    weights = flat(weights)
    rows = logits.reshape(-1, logits.shape[-1])
    # rows may lie further apart than their length; anything else is copied
    if rows.stride(1) != 1 or (len(rows) > 1 and rows.stride(0) < rows.shape[1]):
        rows = rows.contiguous()
    loss = DistillFunction.apply(
        rows, values.reshape(-1, values.shape[-1]).contiguous(),
        indices.reshape(-1, indices.shape[-1]).contiguous(), flat(labels), weights,
        float(temperature), float(label_weight))
    if reduction == "none":
        return loss.reshape(lead)
    if reduction == "sum":
        return loss.sum()
    return loss.sum() / (loss.numel() if weights is None else weights.sum())


class DistillLoss(torch.nn.Module):
    """``distill_loss`` with its temperature, label weight and reduction kept."""

    def __init__(self, temperature=1.0, label_weight=0.0, reduction="mean"):
        super().__init__()
        self.temperature, self.label_weight = float(temperature), float(label_weight)
        self.reduction = reduction

    def forward(self, logits, values, indices, labels=None, weights=None):
        return distill_loss(logits, values, indices, labels, weights, self.temperature,
                            self.label_weight, self.reduction)
