"""The operators of a compressed feed-forward block and of its training, as measured.

- "glu": the gated half of a feed-forward block over sums of Kronecker products,
  h = act(x Wg + bg) * (x Wu + bu), W* = sum_i kron(S* (.) A*_i, B*_i): forward and backward.
- "distill": the loss that recovers a compressed model from its dense original, against the
  original's top logits of each row (temperature, optional hard labels): loss, gradient, and
  both in one call.

With ``own`` false ``run`` computes them in elementary torch operations in float32, with
``own`` true through the package's entry points.
"""
import math

import torch

own = False

# gate and up are stacked: S [2][p][q], A [2][r][p][q], B [2][r][m1][m2], bias [2][q*m2]
ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "sigmoid")


def _glu(name, direction, dtype, N, p, q, m1, m2, r, act, bias=True):
    return {"name": name, "op": "glu", "direction": direction, "dtype": dtype, "N": N, "p": p,
            "q": q, "m1": m1, "m2": m2, "r": r, "act": act, "bias": bias}


def _distill(name, direction, dtype, N, V, K, tau, label_weight):
    return {"name": name, "op": "distill", "direction": direction, "dtype": dtype, "N": N, "V": V,
            "K": K, "tau": tau, "label_weight": label_weight}


def listed():
    return [
        # one token of a serving loop through the tutorial layer's sizes: latency
        _glu("glu_fwd_token", "fwd", "bf16", 1, 32, 32, 32, 32, 4, "silu"),
        # a short ragged prompt, rank one, rectangular blocks at GPT-2 small's width
        _glu("glu_fwd_ragged", "fwd", "bf16", 517, 24, 32, 32, 64, 1, "gelu_tanh"),
        # the tutorial's 20,000 rows
        _glu("glu_fwd_rows", "fwd", "bf16", 20000, 32, 32, 32, 32, 4, "silu"),
        # the large layer (4096 wide, eight terms) on 16 K tokens
        _glu("glu_fwd_large", "fwd", "bf16", 16384, 64, 64, 64, 64, 8, "silu"),
        # exact FP32 on an evaluation batch
        _glu("glu_fwd_f32", "fwd", "f32", 1000, 32, 32, 32, 32, 2, "gelu"),
        # a ragged micro-batch of a fine-tuning step
        _glu("glu_bwd_ragged", "bwd", "bf16", 1021, 24, 32, 32, 64, 2, "gelu_tanh"),
        # the tutorial's training batch
        _glu("glu_bwd_rows", "bwd", "bf16", 20000, 32, 32, 32, 32, 4, "silu"),
        # exact FP32 training at a small odd batch, no bias
        _glu("glu_bwd_f32", "bwd", "f32", 777, 32, 24, 16, 32, 2, "silu", bias=False),
        # the loss of the last positions of a few sequences, GPT-2's odd vocabulary
        _distill("distill_fwd_few", "fwd", "bf16", 3, 50257, 64, 2.0, 0.0),
        # the gradient as autograd asks for it, after the loss
        _distill("distill_bwd", "bwd", "bf16", 1023, 32000, 32, 1.0, 0.5),
        # a training step over 4096 positions: loss and gradient from one call
        _distill("distill_step_tokens", "step", "bf16", 4096, 50257, 64, 2.0, 0.25),
        # float32 logits of a small odd batch
        _distill("distill_step_f32", "step", "f32", 515, 50257, 128, 4.0, 0.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    if rng.random() < 0.6:
        direction = rng.choice(("fwd", "bwd"))
        dtype = "bf16" if rng.random() < 0.75 else "f32"
        if dtype == "bf16":
            p, q, r = rng.randint(8, 64), rng.randint(8, 64), _log_int(rng, 1, 8)
            m1, m2, N = 8 * rng.randint(2, 8), 8 * rng.randint(2, 8), _log_int(rng, 1, 20000)
            most = 200e9
        else:
            p, q, r = rng.randint(4, 32), rng.randint(4, 32), _log_int(rng, 1, 4)
            m1, m2, N = 4 * rng.randint(2, 8), 4 * rng.randint(2, 8), _log_int(rng, 1, 3000)
            most = 8e9
        c = _glu("", direction, dtype, N, p, q, m1, m2, r, rng.choice(ACTIVATIONS),
                 rng.random() < 0.7)
        while work(c)["flops"] > most and c["N"] > 1:
            c["N"] //= 2
    else:
        dtype = rng.choice(("bf16", "bf16", "f32"))
        V, N = _log_int(rng, 1000, 131072), _log_int(rng, 1, 4096)
        N = max(1, min(N, 200_000_000 // (V * (2 if dtype == "bf16" else 4))))
        c = _distill("", rng.choice(("fwd", "bwd", "step")), dtype, N, V, _log_int(rng, 1, 256),
                     rng.choice((1.0, 1.5, 2.0, 4.0)), rng.choice((0.0, 0.25, 0.5, 1.0)))
    del c["name"]
    return c


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    N = c["N"]
    if c["op"] == "glu":
        p, q, m1, m2, r = (c[k] for k in ("p", "q", "m1", "m2", "r"))
        factors = 2 * e * (p * q + r * p * q + r * m1 * m2 + q * m2)
        # multiply-adds per row and term in the cheaper contraction order
        macs = min(p * m1 * m2 + p * q * m2, p * q * m1 + q * m1 * m2)
        forward = 2 * 2 * r * macs * N
        if c["direction"] == "fwd":
            return {"bytes": e * N * (p * m1 + q * m2) + factors, "flops": forward}
        # both pre-activations again, dX, and the factors' gradients
        return {"bytes": e * N * (2 * p * m1 + q * m2) + 2 * factors, "flops": 3 * forward}
    V, K = c["V"], c["K"]
    logits = N * V * e
    rows = N * K * 12 + N * 16
    if c["direction"] == "fwd":
        return {"bytes": logits + rows, "flops": 3 * N * V}
    return {"bytes": 2 * logits + rows, "flops": (3 if c["direction"] == "bwd" else 6) * N * V}


# ---- inputs -------------------------------------------------------------------------


def _prepare_glu(c, gen, dev, t):
    N, p, q, m1, m2, r = (c[k] for k in ("N", "p", "q", "m1", "m2", "r"))
    rand = lambda *s: torch.randn(*s, device=dev, generator=gen)  # noqa: E731
    s = {"x": rand(N, p * m1).to(t),
         # half of S zero, as an l1-trained layer has it
         "S": (torch.rand(2, p, q, device=dev, generator=gen) < 0.5).to(t),
         "A": (rand(2, r, p, q) / math.sqrt(p)).to(t),
         "B": (rand(2, r, m1, m2) / math.sqrt(m1)).to(t),
         "bias": (0.1 * rand(2, q * m2)).to(t) if c["bias"] else None}
    if c["direction"] == "bwd":
        s["dH"] = rand(N, q * m2).to(t)
    return s


def _prepare_distill(c, gen, dev, t):
    N, V, K = c["N"], c["V"], c["K"]
    logits = torch.empty(N, V, device=dev, dtype=t)
    values = torch.empty(N, K, device=dev)
    indices = torch.empty(N, K, device=dev, dtype=torch.int64)
    for a in range(0, N, 512):
        b = min(N, a + 512)
        z = 2.5 * torch.randn(b - a, V, device=dev, generator=gen)
        logits[a:b] = z.to(t)
        # the teacher agrees with the student up to noise
        values[a:b], indices[a:b] = (z + torch.randn(b - a, V, device=dev, generator=gen)).topk(K)
    # some rows keep fewer than K entries; the first keeps all of them
    short = torch.rand(N, device=dev, generator=gen) < 0.1
    short[0] = False
    cut = torch.randint(1, K + 1, (N,), device=dev, generator=gen)
    gone = short[:, None] & (torch.arange(K, device=dev)[None] >= cut[:, None])
    indices[gone] = -1
    values[gone] = float("nan")
    labels = torch.randint(0, V, (N,), device=dev, generator=gen)
    labels[1:][torch.rand(N - 1, device=dev, generator=gen) < 0.05] = -100
    # the weight of each row in the batch's mean; padding has none
    weights = torch.ones(N, device=dev)
    weights[1:][torch.rand(N - 1, device=dev, generator=gen) < 0.1] = 0.0
    weights /= weights.sum()
    return {"logits": logits, "values": values, "indices": indices, "labels": labels,
            "weights": weights}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = (_prepare_glu if case["op"] == "glu" else _prepare_distill)(case, gen, dev, t)
    s["case"] = case
    if case["op"] == "distill" and case["direction"] == "bwd":
        # what the forward call left for the gradient: the log-sum-exp of each row at the
        # temperature and at one
        s["lse"] = torch.stack([_lse(s["logits"].float() / case["tau"])[:, 0],
                                _lse(s["logits"].float())[:, 0]], 1)
    return s


# ---- plain forms ---------------------------------------------------------------------


def _lse(z):
    m = z.max(1, keepdim=True).values
    return m + (z - m).exp().sum(1, keepdim=True).log()


def _act(g, name):
    """act(g) and its derivative."""
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(g / math.sqrt(2)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        th = torch.tanh(k * (g + 0.044715 * g * g * g))
        return (0.5 * g * (1 + th),
                0.5 * (1 + th) + 0.5 * g * (1 - th * th) * k * (1 + 3 * 0.044715 * g * g))
    sg = 1 / (1 + torch.exp(-g))
    if name == "sigmoid":
        return sg, sg * (1 - sg)
    return g * sg, sg + g * sg * (1 - sg)


def _mix(X, B):
    """X [N][p][j] against B [r][j][k]: T [N][k][r*p]."""
    N, p, j = X.shape
    r, _, k = B.shape
    T = X.reshape(N * p, j) @ B.permute(1, 0, 2).reshape(j, r * k)
    return T.reshape(N, p, r, k).permute(0, 3, 2, 1).reshape(N, k, r * p)


def _project(x, C, B, bias):
    """x sum_i kron(C_i, B_i) + bias, by the vec trick."""
    r, p, q = C.shape
    T = _mix(x.reshape(x.shape[0], p, -1), B)
    y = (T @ C.reshape(r * p, q)).transpose(1, 2).reshape(x.shape[0], -1)
    return y if bias is None else y + bias


def _project_back(x, C, B, dy):
    """(dx, dC, dB) of one projection."""
    r, p, q = C.shape
    _, m1, m2 = B.shape
    N = x.shape[0]
    G = dy.reshape(N, q, m2)
    X = x.reshape(N, p, m1)
    T = _mix(X, B).reshape(N * m2, r * p)
    dC = (T.t() @ G.transpose(1, 2).reshape(N * m2, q)).reshape(r, p, q)
    # U[n][a][(i,k)] = sum_c C_i[a][c] G[n][c][k]
    U = G.transpose(1, 2).reshape(N * m2, q) @ C.permute(2, 0, 1).reshape(q, r * p)
    U = U.reshape(N, m2, r, p).permute(0, 3, 2, 1).reshape(N * p, r * m2)
    dB = (X.reshape(N * p, m1).t() @ U).reshape(m1, r, m2).permute(1, 0, 2)
    dx = (U @ B.permute(0, 2, 1).reshape(r * m2, m1)).reshape(N, p * m1)
    return dx, dC, dB


def _plain_glu(s):
    c = s["case"]
    t = s["x"].dtype
    x, S, A, B = (s[k].float() for k in ("x", "S", "A", "B"))
    b = [None, None] if s["bias"] is None else s["bias"].float()
    C = S[:, None] * A
    g, u = _project(x, C[0], B[0], b[0]), _project(x, C[1], B[1], b[1])
    f, df = _act(g, c["act"])
    if c["direction"] == "fwd":
        return (f * u).to(t)
    dH = s["dH"].float()
    du, dg = dH * f, dH * u * df
    gx, gC, gB = _project_back(x, C[0], B[0], dg)
    ux, uC, uB = _project_back(x, C[1], B[1], du)
    dC = torch.stack([gC, uC])
    out = {"dX": gx + ux, "dS": (dC * A).sum(1), "dA": dC * S[:, None],
           "dB": torch.stack([gB, uB])}
    if s["bias"] is not None:
        out["dbias"] = torch.stack([dg.sum(0), du.sum(0)])
    return {k: v.to(t) for k, v in out.items()}


def _plain_distill(s):
    c = s["case"]
    tau, lam = c["tau"], c["label_weight"]
    x = s["logits"].float()
    N, V = x.shape
    there = s["indices"] >= 0
    idx = s["indices"].clamp(min=0)
    v = torch.where(there, s["values"], float("-inf")) / tau
    logp = v - _lse(v)
    p = logp.exp()
    hard = (s["labels"] >= 0).float()
    lab = s["labels"].clamp(min=0)[:, None]
    w = s["weights"][:, None]
    out = {}
    if c["direction"] == "bwd":
        lse_t, lse_1 = s["lse"][:, :1], s["lse"][:, 1:]
    else:
        lse_t, lse_1 = _lse(x / tau), _lse(x)
        logq = x.gather(1, idx) / tau - lse_t
        kl = torch.where(there, p * (logp - logq), 0.0).sum(1, keepdim=True)
        ce = (lse_1 - x.gather(1, lab)) * hard[:, None]
        out["loss"] = (w * ((1 - lam) * tau * tau * kl + lam * ce))[:, 0]
    if c["direction"] != "fwd":
        d = (1 - lam) * tau * (x / tau - lse_t).exp()
        d.scatter_add_(1, idx, torch.where(there, -(1 - lam) * tau * p, 0.0))
        if lam:
            d += lam * hard[:, None] * (x - lse_1).exp()
            d.scatter_add_(1, lab, -lam * hard[:, None])
        out["dlogits"] = (w * d).to(s["logits"].dtype)
    return out


# ---- the definitions in 64 bits, written another way -------------------------------------


def _exact_act(g, name):
    if name == "silu":
        f = lambda v: v * torch.sigmoid(v)  # noqa: E731
    elif name == "sigmoid":
        f = torch.sigmoid
    elif name == "gelu":
        f = lambda v: v * torch.special.ndtr(v)  # noqa: E731
    else:
        f = lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi)  # noqa: E731
                                        * (v + 0.044715 * v ** 3))
    v = g.detach().requires_grad_(True)
    with torch.enable_grad():
        y = f(v)
        (d,) = torch.autograd.grad(y.sum(), v)
    return y.detach(), d


def _exact_glu(s):
    """Builds both dense matrices and their dense gradients."""
    c = s["case"]
    p, q, m1, m2, r = (c[k] for k in ("p", "q", "m1", "m2", "r"))
    x, S, A, B = (s[k].double() for k in ("x", "S", "A", "B"))
    W = [sum(torch.kron(S[k] * A[k, i], B[k, i]) for i in range(r)) for k in (0, 1)]
    y = [x @ w for w in W]
    if s["bias"] is not None:
        y = [v + s["bias"][k].double() for k, v in enumerate(y)]
    f, df = _exact_act(y[0], c["act"])
    if c["direction"] == "fwd":
        return f * y[1]
    dH = s["dH"].double()
    d = [dH * y[1] * df, dH * f]
    out = {"dX": d[0] @ W[0].t() + d[1] @ W[1].t()}
    dS, dA, dB = torch.zeros_like(S), torch.zeros_like(A), torch.zeros_like(B)
    for k in (0, 1):
        dW = (x.t() @ d[k]).reshape(p, m1, q, m2)
        for i in range(r):
            dC = torch.einsum("ajck,jk->ac", dW, B[k, i])
            dS[k] += dC * A[k, i]
            dA[k, i] = dC * S[k]
            dB[k, i] = torch.einsum("ajck,ac->jk", dW, S[k] * A[k, i])
    out |= {"dS": dS, "dA": dA, "dB": dB}
    if s["bias"] is not None:
        out["dbias"] = torch.stack([v.sum(0) for v in d])
    return out


def _exact_distill(s):
    """The gradient by automatic differentiation of the loss's definition, some rows at a time."""
    c = s["case"]
    tau, lam = c["tau"], c["label_weight"]
    losses, grads = [], []
    for a in range(0, c["N"], 512):
        z = s["logits"][a:a + 512].double().requires_grad_(True)
        there = s["indices"][a:a + 512] >= 0
        target = torch.zeros_like(z)
        v = s["values"][a:a + 512].double().masked_fill(~there, float("-inf"))
        target.scatter_add_(1, s["indices"][a:a + 512].clamp(min=0), torch.softmax(v / tau, 1))
        with torch.enable_grad():
            logq = torch.log_softmax(z / tau, 1)
            loss = (1 - lam) * tau ** 2 * (torch.xlogy(target, target) - target * logq).sum(1)
            loss = loss + lam * torch.nn.functional.cross_entropy(
                z, s["labels"][a:a + 512], ignore_index=-100, reduction="none")
            loss = loss * s["weights"][a:a + 512].double()
            (g,) = torch.autograd.grad(loss.sum(), z)
        losses.append(loss.detach())
        grads.append(g.to(torch.float64))
    out = {} if c["direction"] == "bwd" else {"loss": torch.cat(losses)}
    if c["direction"] != "fwd":
        out["dlogits"] = torch.cat(grads)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_glu if case["op"] == "glu" else _exact_distill)(s)


# ---- one pass ------------------------------------------------------------------------


def _own_glu(s):
    from kronecker_factored_structured_b200 import native

    c = s["case"]
    if c["direction"] == "fwd":
        return native.glu_forward(s["x"], s["S"], s["A"], s["B"], s["bias"], activation=c["act"],
                                  dtype=c["dtype"])
    g = native.glu_backward(s["x"], s["S"], s["A"], s["B"], s["dH"], s["bias"],
                            activation=c["act"], dtype=c["dtype"],
                            need_dbias=s["bias"] is not None)
    return {k: v for k, v in g.items() if v is not None}


def _own_distill(s):
    from kronecker_factored_structured_b200 import native

    c = s["case"]
    kw = dict(labels=s["labels"], temperature=c["tau"], label_weight=c["label_weight"])
    args = (s["logits"], s["values"], s["indices"])
    if c["direction"] == "fwd":
        return {"loss": native.distill_forward(*args, weights=s["weights"], **kw)["loss"]}
    if c["direction"] == "bwd":
        return {"dlogits": native.distill_backward(*args, s["lse"], weights=s["weights"], **kw)}
    g = native.distill_step(*args, weights=s["weights"], **kw)
    return {"loss": g["loss"], "dlogits": g["dlogits"]}


def run(state):
    if own:
        return (_own_glu if state["case"]["op"] == "glu" else _own_distill)(state)
    return (_plain_glu if state["case"]["op"] == "glu" else _plain_distill)(state)
