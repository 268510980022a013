"""The gated half h = act(x Wg + bg) * (x Wu + bu) in 64 bits through the dense matrices, with
bounds on what the BF16 kernels' roundings may add, term by term.

One rounding to bfloat16 moves a value by at most U = 2^-8 of itself.  The kernels round
C = S (.) A once (nothing where S is 0 or 1, counted all the same), T = X B, and the gradients
dg, du of the pre-activations, and their outputs; the product V = dg B^T on the way to dX as T.
With M the product of absolute values that a rounded factor enters, the bounds below are
    |g|: 2 U sum |C| |X B|,   |dX|: sum |C| (|d| bounds |B|) + 2 U sum |C| |d B^T|, ...
and 2^-12 of each sum of absolute values covers fp32 accumulation and the hardware
exponentials (chains of up to 2^9 terms of 2^-24, 2^-21 per activation)."""
import math

import torch

U = 2.0 ** -8
ACC = 2.0 ** -12


def act(g, name):
    g = g.detach().requires_grad_(True)
    with torch.enable_grad():
        if name == "silu":
            f = g * torch.sigmoid(g)
        elif name == "gelu":
            f = g * torch.special.ndtr(g)
        elif name == "gelu_tanh":
            f = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
        else:
            f = torch.sigmoid(g)
        (d,) = torch.autograd.grad(f.sum(), g)
    return f.detach(), d


def _sum_kron(C, B):
    return sum(torch.kron(C[i], B[i]) for i in range(C.shape[0]))


def reference(d, name):
    """{output: (value, bound)}; gradients where d holds dH."""
    x, S, A, B = (d[k].double() for k in ("x", "S", "A", "B"))
    two, r, p, q = A.shape
    m1, m2 = B.shape[2:]
    N = x.shape[0]
    C = S[:, None] * A
    W = [_sum_kron(C[k], B[k]) for k in (0, 1)]
    b = d.get("bias")
    y, e = [], []
    for k in (0, 1):
        y.append(x @ W[k] + (b[k].double() if b is not None else 0.0))
        T = torch.einsum("naj,ijk->niak", x.view(N, p, m1), B[k]).abs()
        Ta = torch.einsum("naj,ijk->niak", x.abs().view(N, p, m1), B[k].abs())
        m = torch.einsum("niak,iac->nck", 2 * U * T + ACC * Ta, C[k].abs())
        e.append(m.reshape(N, q * m2) + ACC * y[k].abs())
    f, df = act(y[0], name)
    eg, eu = e
    ef = 1.2 * eg + ACC * f.abs()          # |act'| <= 1.13
    h = f * y[1]
    out = {"h": (h, ef * (y[1].abs() + eu) + f.abs() * eu + U * h.abs())}
    if "dH" not in d:
        return out
    dH = d["dH"].double()
    dd = [dH * y[1] * df, dH * f]
    # |act''| <= 0.8
    ed = [dH.abs() * (eu * (df.abs() + 0.8 * eg) + y[1].abs() * (0.8 * eg + ACC))
          + U * dd[0].abs(), dH.abs() * ef + U * dd[1].abs()]
    dX = dd[0] @ W[0].t() + dd[1] @ W[1].t()
    eX = U * dX.abs()
    vals = {k: [] for k in ("dS", "dA", "dB", "dbias")}
    errs = {k: [] for k in vals}
    for k in (0, 1):
        Wa = _sum_kron(C[k].abs(), B[k].abs())
        V = torch.einsum("nck,ijk->nicj", dd[k].view(N, q, m2), B[k]).abs()
        m = torch.einsum("nicj,iac->naj", 2 * U * V, C[k].abs())
        eX += (ed[k] + ACC * dd[k].abs()) @ Wa.t() + m.reshape(N, p * m1)
        dW = (x.t() @ dd[k]).view(p, m1, q, m2)
        eW = (x.abs().t() @ (ed[k] + ACC * dd[k].abs())).view(p, m1, q, m2) + ACC * dW.abs()
        dC = torch.einsum("ajck,ijk->iac", dW, B[k])
        eC = torch.einsum("ajck,ijk->iac", eW + ACC * dW.abs(), B[k].abs())
        dB = torch.einsum("ajck,iac->ijk", dW, C[k])
        eB = torch.einsum("ajck,iac->ijk", eW + ACC * dW.abs(), C[k].abs())
        one = {"dS": ((dC * A[k]).sum(0), (eC * A[k].abs()).sum(0)),
               "dA": (dC * S[k], eC * S[k].abs()), "dB": (dB, eB),
               "dbias": (dd[k].sum(0), (ed[k] + ACC * dd[k].abs()).sum(0))}
        for n, (v, er) in one.items():
            vals[n].append(v)
            errs[n].append(er + U * v.abs())
    out["dX"] = (dX, eX)
    for n in vals:
        out[n] = (torch.stack(vals[n]), torch.stack(errs[n]))
    return out
