"""GPU tests of the distillation loss (kron_distill_forward / _backward / _step through the
binding) against its definition in 64 bits on the CPU.

Tolerances.  An exponent (x - m)/tau log2(e) of size up to about 60 carries two fp32 roundings
(60 * 2 * 2^-24 = 7e-6), the hardware's ex2 2^-22, and a sum of up to 2^17 terms, in chains of
at most 2^8 per thread and 2^5 across threads, 290 * 2^-24 = 1.7e-5: a probability is off by at
most 3e-5 of itself, a log-sum-exp by 3e-5 plus a rounding of its own size.  A bfloat16
gradient adds half a step, 2^-8 of itself."""
import pytest
import torch

import kronecker_factored_structured_b200 as kfs
from kronecker_factored_structured_b200 import native

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
EPS = 3e-5
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def make(N, V, K, dtype, seed, idx=torch.int64, pad=0, offset=0, scale=3.0, duplicates=False,
         holes=True):
    g = torch.Generator().manual_seed(seed)
    x = (scale * torch.randn(N, V, generator=g)).to(dtype)
    store = torch.full((N * (V + pad) + offset,), float("nan"), dtype=dtype)
    rows = store[offset:].view(N, V + pad)[:, :V]
    rows.copy_(x)
    t = x.float() + torch.randn(N, V, generator=g)
    if duplicates:
        i = torch.randint(0, min(V, 5), (N, K), generator=g)
        v = torch.gather(t, 1, i) + torch.randn(N, K, generator=g)
    else:
        v, i = t.topk(K)
    labels = torch.randint(0, V, (N,), generator=g)
    w = torch.rand(N, generator=g) + 0.5
    if holes:
        if N > 1:
            i[1] = -1                       # a row without entries, its values not to be read
            v[1] = float("nan")
        if N > 2:
            labels[2] = -100
            i[2, 0] = V                     # outside: no entry
        if N > 3:
            w[3] = 0.0
        if N > 4 and K > 1:
            v[4, 0] = float("-inf")
        if N > 5:
            v[5] = float("-inf")            # nothing with a weight
    d = {"logits": store, "values": v, "indices": i.to(idx), "labels": labels, "weights": w}
    d = {k: t.to(DEV) for k, t in d.items()}
    d["logits"] = d["logits"][offset:].view(N, V + pad)[:, :V]
    return d


def reference(d, tau, lam, dloss=None):
    """(loss, dlogits, scale of each gradient entry) in 64 bits, on the CPU."""
    x = d["logits"].double().cpu()
    N, V = x.shape
    i, v = d["indices"].long().cpu(), d["values"].double().cpu()
    there = (i >= 0) & (i < V)
    v = torch.where(there, v, float("-inf"))
    some = (v > float("-inf")).any(1, keepdim=True)
    p = torch.where(some, torch.softmax(torch.where(some, v, 0.0) / tau, 1), 0.0)
    P = torch.zeros_like(x).scatter_add_(1, torch.where(there, i, 0), torch.where(there, p, 0.0))
    logp = torch.log_softmax(torch.where(some, v, 0.0) / tau, 1)
    logq = torch.log_softmax(x / tau, 1)
    terms = p * (logp - torch.gather(logq, 1, torch.where(there, i, 0)))
    kl = torch.where(p > 0, terms, 0.0).sum(1)
    lab = d["labels"].cpu() if d["labels"] is not None else torch.full((N,), -1)
    has = (lab >= 0) & (lab < V)
    at = torch.where(has, lab, 0)[:, None]
    ce = torch.where(has, -torch.log_softmax(x, 1).gather(1, at)[:, 0], 0.0)
    w = torch.ones(N).double() if d["weights"] is None else d["weights"].double().cpu()
    loss = w * ((1 - lam) * tau ** 2 * kl + lam * ce)
    onehot = torch.zeros_like(x).scatter_(1, at, has.double()[:, None])
    soft = (1 - lam) * tau
    q, s1 = logq.exp() * some, torch.softmax(x, 1) * has[:, None]
    c = (w if dloss is None else w * dloss.double().cpu())[:, None]
    grad = c * (soft * (q - P) + lam * (s1 - onehot))
    size = c.abs() * (soft * (q + P) + lam * (s1 + onehot))
    on = (c != 0)
    loss = torch.where(w != 0, loss, 0.0)
    return loss, torch.where(on, grad, 0.0), torch.where(on, size, 0.0)


def check_loss(got, ref, d, tau, lam):
    # |log p - log q| of the entries is bounded by the logits' range over tau plus log V
    x = d["logits"].double()
    span = float((x.max() - x.min()) / tau + 20)
    w = 1.0 if d["weights"] is None else d["weights"].double().cpu()
    tol = w * EPS * ((1 - lam) * tau ** 2 * (2 + span) + lam * (2 + span * tau))
    assert got.dtype == torch.float32
    assert ((got.double().cpu() - ref).abs() <= tol).all(), (got.cpu(), ref)


def check_grad(got, ref, size, dtype):
    assert got.dtype == dtype
    err = (got.double().cpu() - ref).abs()
    tol = EPS * size + HALF[dtype] * ref.abs() + 1e-37
    assert (err <= tol).all(), float((err - tol).max())


KW = dict(temperature=1.0, label_weight=0.0)
MODES = [(1.0, 0.0), (1.0, 0.4), (2.0, 0.3), (4.0, 0.25), (1.5, 0.5), (3.0, 0.0), (2.0, 1.0)]
# a warp per row (up to 1024 columns and 64 entries) and a CTA per row, on both sides of the edge
SHAPES = [(13, 1024, 64), (13, 1025, 64), (13, 1024, 65), (2001, 10, 5), (1, 1, 1), (7, 2, 2),
          (6, 7, 3), (9, 10, 5), (8, 257, 64), (6, 1000, 300),
          (7, 4096, 1), (3, 50257, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "N{}_V{}_K{}".format(*s))
def test_shapes(shape, dtype):
    for k, (tau, lam) in enumerate(MODES):
        d = make(*shape, dtype, seed=k)
        ref, grad, size = reference(d, tau, lam)
        kw = dict(labels=d["labels"], weights=d["weights"], temperature=tau, label_weight=lam)
        args = (d["logits"], d["values"], d["indices"])
        f = native.distill_forward(*args, **kw)
        check_loss(f["loss"], ref, d, tau, lam)
        check_grad(native.distill_backward(*args, f["lse"], **kw), grad, size, dtype)
        s = native.distill_step(*args, **kw)
        assert torch.equal(s["loss"], f["loss"])
        check_grad(s["dlogits"], grad, size, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1021, 3001])
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (7, 5), (8, 0)])
def test_strided_and_misaligned_rows(pad, offset, V, dtype):
    N, K = 9, 17
    d = make(N, V, K, dtype, seed=3, pad=pad, offset=offset, idx=torch.int32)
    ref, grad, size = reference(d, 2.0, 0.3)
    kw = dict(labels=d["labels"], weights=d["weights"], temperature=2.0, label_weight=0.3)
    args = (d["logits"], d["values"], d["indices"])
    s = native.distill_step(*args, **kw)
    check_loss(s["loss"], ref, d, 2.0, 0.3)
    check_grad(s["dlogits"], grad, size, dtype)
    # into rows of another stride: what lies between them stays as it was
    wide = torch.full((N, V + 5), 7.0, dtype=dtype, device=DEV)
    native.distill_step(*args, out=wide[:, :V], **kw)
    assert torch.equal(wide[:, :V], s["dlogits"]) and bool((wide[:, V:] == 7.0).all())


@pytest.mark.parametrize("step", [False, True])
def test_in_place(step):
    d = make(8, 3001, 40, torch.bfloat16, seed=5)
    kw = dict(labels=d["labels"], weights=d["weights"], temperature=2.0, label_weight=0.3)
    args = (d["logits"], d["values"], d["indices"])
    want = native.distill_step(*args, **kw)
    own = d["logits"].clone()
    if step:
        got = native.distill_step(own, *args[1:], out=own, **kw)
        assert torch.equal(got["loss"], want["loss"]) and got["dlogits"] is own
    else:
        lse = native.distill_forward(*args, **kw)["lse"]
        want = {"dlogits": native.distill_backward(*args, lse, **kw)}
        native.distill_backward(own, *args[1:], lse, out=own, **kw)
    assert torch.equal(own, want["dlogits"])


@pytest.mark.parametrize("V", [300, 3000])
def test_columns_listed_more_than_once(V):
    for dtype in (torch.float32, torch.bfloat16):
        d = make(10, V, 33, dtype, seed=6, duplicates=True)
        d["labels"][6] = int(d["indices"][6, 0])     # the label is one of them
        for tau, lam in ((1.0, 0.0), (2.0, 0.5)):
            ref, grad, size = reference(d, tau, lam)
            s = native.distill_step(d["logits"], d["values"], d["indices"], labels=d["labels"],
                                    weights=d["weights"], temperature=tau, label_weight=lam)
            check_loss(s["loss"], ref, d, tau, lam)
            # a column's share is a sum of up to K probabilities
            check_grad(s["dlogits"], grad, 2 * size, dtype)


def test_most_entries():
    d = make(4, 5000, 1024, torch.bfloat16, seed=7)
    ref, grad, size = reference(d, 1.0, 0.0)
    s = native.distill_step(d["logits"], d["values"], d["indices"], weights=d["weights"])
    check_loss(s["loss"], ref, d, 1.0, 0.0)
    check_grad(s["dlogits"], grad, size, torch.bfloat16)


@pytest.mark.parametrize("V", [999, 1999])
def test_infinities_and_nan(V):
    """-inf logits have probability zero; a row of weight zero is zero whatever it holds; a NaN
    shows in its own row only."""
    d = make(6, V, 8, torch.float32, seed=8, holes=False)
    x = d["logits"]
    x[0, 500:] = float("-inf")
    d["indices"][0] = torch.arange(8, device=DEV)
    x[0, 499] = float("-inf")
    x[1, 3] = float("nan")
    x[2] = float("nan")
    d["weights"][2] = 0.0
    x[3, :V - 1] = -3e38
    x[4] = float("-inf")
    d["weights"][4] = 0.0
    kw = dict(labels=d["labels"], weights=d["weights"], temperature=2.0, label_weight=0.0)
    s = native.distill_step(x, d["values"], d["indices"], **kw)
    ref, grad, size = reference(d, 2.0, 0.0)
    assert bool(torch.isnan(s["loss"][1])) and bool(torch.isnan(s["dlogits"][1]).any())
    for r in (0, 2, 4, 5):
        one = {k: v[r:r + 1] for k, v in d.items()}
        lo, gr, si = reference(one, 2.0, 0.0)
        if r in (2, 4):
            assert float(s["loss"][r]) == 0.0 and not s["dlogits"][r].any()
        else:
            one["logits"] = one["logits"].nan_to_num(neginf=-60)
            check_loss(s["loss"][r:r + 1], lo, one, 2.0, 0.0)
            check_grad(s["dlogits"][r:r + 1], gr, si, torch.float32)
    assert not s["dlogits"][0, 500:].any()
    # an entry on a column of probability zero: infinite loss, as the definition has it
    d["indices"][0, 0] = 600
    assert float(native.distill_step(x, d["values"], d["indices"], **kw)["loss"][0]) == float("inf")


def test_large_logits():
    d = make(5, 2000, 16, torch.float32, seed=9, scale=2000.0, holes=False)
    for tau, lam in ((1.0, 0.0), (2.0, 0.5), (1.5, 0.5)):
        ref, grad, size = reference(d, tau, lam)
        s = native.distill_step(d["logits"], d["values"], d["indices"], labels=d["labels"],
                                weights=d["weights"], temperature=tau, label_weight=lam)
        # exponents of size 1e4 round to 1e4 * 2^-23 = 1e-3 of the probability
        assert torch.allclose(s["loss"].double().cpu(), ref, rtol=3e-5)
        err = (s["dlogits"].double().cpu() - grad).abs()
        assert (err <= 2e-3 * size + 1e-6).all()


def test_gradient_against_differences():
    d = make(4, 37, 6, torch.float32, seed=10, holes=False, scale=1.0)
    kw = dict(labels=d["labels"], weights=d["weights"], temperature=1.5, label_weight=0.4)
    x = d["logits"].clone()
    g = native.distill_step(x, d["values"], d["indices"], **kw)["dlogits"].double().cpu()
    h = 2.0 ** -4
    for v in range(0, 37, 5):
        lo, hi = x.clone(), x.clone()
        lo[:, v] -= h
        hi[:, v] += h
        f = [native.distill_forward(t, d["values"], d["indices"], **kw)["loss"].double().cpu()
             for t in (lo, hi)]
        # h^2/6 times a third derivative below 1, and 2 * 1e-5 / 2h of rounding
        assert ((f[1] - f[0]) / (2 * h) - g[:, v]).abs().max() <= h * h / 6 * 1.5 + 3e-4


def test_autograd_reductions_and_leading_dims():
    d = make(12, 501, 9, torch.bfloat16, seed=11)
    z = d["logits"].reshape(3, 4, 501).clone().requires_grad_(True)
    sh = lambda k: d[k].reshape(3, 4, *d[k].shape[1:])  # noqa: E731
    ref, grad, size = reference(d, 2.0, 0.3)
    total = float(d["weights"].double().sum())
    for red, c in (("sum", 1.0), ("mean", 1 / total), ("none", 1.0)):
        loss = kfs.distill_loss(z, sh("values"), sh("indices"), sh("labels"), sh("weights"),
                                temperature=2.0, label_weight=0.3, reduction=red)
        if red == "none":
            assert loss.shape == (3, 4)
            loss = loss.sum()
        (g,) = torch.autograd.grad(loss, z)
        assert abs(float(loss) - c * float(ref.sum())) <= 1e-4 * (1 + c * float(ref.abs().sum()))
        check_grad(g.reshape(12, 501), c * grad, 2 * c * size, torch.bfloat16)
    loss = kfs.DistillLoss(2.0, 0.3)(z, sh("values"), sh("indices"), sh("labels"), sh("weights"))
    assert abs(float(loss) - float(ref.sum()) / total) <= 1e-4 * (1 + float(ref.abs().sum()))


def test_upstream_gradient_per_row():
    d = make(8, 777, 9, torch.float32, seed=12)
    up = torch.randn(8, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    up[5] = 0.0
    kw = dict(labels=d["labels"], weights=d["weights"], temperature=4.0, label_weight=0.2)
    args = (d["logits"], d["values"], d["indices"])
    lse = native.distill_forward(*args, **kw)["lse"]
    _, grad, size = reference(d, 4.0, 0.2, up)
    check_grad(native.distill_backward(*args, lse, up, **kw), grad, size, torch.float32)


def test_no_rows():
    d = {"logits": torch.empty(0, 10, device=DEV), "values": torch.empty(0, 3, device=DEV),
         "indices": torch.empty(0, 3, dtype=torch.int64, device=DEV)}
    s = native.distill_step(**d)
    assert s["loss"].shape == (0,) and s["dlogits"].shape == (0, 10)


def test_rows_beyond_32_bits():
    """70,001 rows of 32,771 columns: offsets pass 2^31 elements.  Rows of weight zero are not
    read, so only the last ones have to be filled."""
    N, V, K = 70001, 32771, 4
    x = torch.empty(N, V, dtype=torch.bfloat16, device=DEV)
    d = make(3, V, K, torch.bfloat16, seed=13, holes=False)
    x[-3:] = d["logits"]
    w = torch.zeros(N, device=DEV)
    w[-3:] = d["weights"]
    v = torch.zeros(N, K, device=DEV)
    i = torch.zeros(N, K, dtype=torch.int64, device=DEV)
    v[-3:], i[-3:] = d["values"], d["indices"]
    s = native.distill_step(x, v, i, weights=w, out=x)
    ref, grad, size = reference(d, 1.0, 0.0)
    check_loss(s["loss"][-3:], ref, d, 1.0, 0.0)
    check_grad(x[-3:], grad, size, torch.bfloat16)
    assert not s["loss"][:-3].any() and not x[:1000].any() and not x[-2000:-3].any()


def test_stream_graph_and_repeat():
    d = make(64, 5003, 32, torch.bfloat16, seed=14)
    kw = dict(labels=d["labels"], weights=d["weights"], temperature=2.0, label_weight=0.3)
    args = (d["logits"], d["values"], d["indices"])
    want = native.distill_step(*args, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = native.distill_step(*args, **kw)
    b = native.distill_step(*args, **kw)
    torch.cuda.synchronize()
    for got in (a, b):
        assert torch.equal(got["loss"], want["loss"])
        assert torch.equal(got["dlogits"], want["dlogits"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = native.distill_step(*args, **kw)
    other = make(64, 5003, 32, torch.bfloat16, seed=15)
    for k in d:
        d[k].copy_(other[k])
    graph.replay()
    fresh = native.distill_step(*args, **kw)
    torch.cuda.synchronize()
    assert torch.equal(c["loss"], fresh["loss"]) and torch.equal(c["dlogits"], fresh["dlogits"])


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_gradient_of_the_weights(reduction):
    """The rows' weights are differentiable: dloss times the loss of the row, and for "mean" the
    denominator's part; a row of weight zero has one too."""
    d = make(8, 777, 9, torch.float32, seed=16, holes=False)
    d["weights"][3] = 0.0
    tau, lam = 2.0, 0.3
    rows, _, _ = reference(dict(d, weights=None), tau, lam)
    w = d["weights"].double().cpu()
    up = torch.randn(8, generator=torch.Generator().manual_seed(2))
    leaf = d["weights"].clone().requires_grad_(True)
    z = d["logits"].clone().requires_grad_(True)
    loss = kfs.distill_loss(z, d["values"], d["indices"], d["labels"], leaf, temperature=tau,
                            label_weight=lam, reduction=reduction)
    if reduction == "none":
        loss = (loss * up.to(DEV)).sum()
    g, gz = torch.autograd.grad(loss, (leaf, z))
    W = w.sum()
    want = {"none": up.double() * rows, "sum": rows,
            "mean": rows / W - (w * rows).sum() / W ** 2}[reduction]
    # a row's loss as in check_loss; "mean" takes a sum over eight rows besides
    x = d["logits"].double()
    span = float((x.max() - x.min()) / tau + 20)
    row_tol = EPS * ((1 - lam) * tau ** 2 * (2 + span) + lam * (2 + span * tau))
    c = {"none": float(up.abs().max()), "sum": 1.0, "mean": 2 / float(W)}[reduction]
    assert g.shape == leaf.shape and g.dtype == torch.float32
    assert float((g.double().cpu() - want).abs().max()) <= c * (row_tol + 16 * 2.0 ** -24 *
                                                                float(rows.abs().max()))
    _, grad, size = reference(d, tau, lam, up if reduction == "none" else None)
    c = 1 / W if reduction == "mean" else 1.0
    check_grad(gz, c * grad, 2 * c * size, torch.float32)


@pytest.mark.parametrize("V", [999, 1999])
@pytest.mark.parametrize("lam", [0.0, 0.4, 1.0])
def test_rows_without_any_term(lam, V):
    """No entries, and no label where the labels count: the row's loss is the constant zero, and
    its gradient is zero whatever its logits hold."""
    for dtype in (torch.float32, torch.bfloat16):
        d = make(6, V, 8, dtype, seed=17, holes=False)
        x = d["logits"]
        x[0, 5], x[1, 7], x[2] = float("nan"), float("inf"), float("-inf")
        x[4, 9] = float("nan")
        d["labels"][:4] = -100
        d["indices"][:3] = -1
        d["values"][3] = float("-inf")               # entries without weight are none
        if lam == 1.0:
            d["indices"][:4] = d["indices"][5]       # entries do not count
            d["values"][:4] = d["values"][5]
        d["weights"][0] = 3.0
        kw = dict(labels=d["labels"], weights=d["weights"], temperature=2.0, label_weight=lam)
        args = (x, d["values"], d["indices"])
        f = native.distill_forward(*args, **kw)
        s = native.distill_step(*args, **kw)
        b = native.distill_backward(*args, f["lse"], **kw)
        for loss, grad in ((s["loss"], s["dlogits"]), (f["loss"], b)):
            assert not loss[:4].any() and not grad[:4].any()
            # a row that has a term still shows its NaN; the one behind it is as ever
            assert bool(loss[4].isnan()) and bool(grad[4].isnan().any())
            assert bool(loss[5].isfinite()) and bool(grad[5].isfinite().all())


@pytest.mark.parametrize("V", [300, 3000])
def test_weight_zero_meets_an_infinite_upstream_gradient(V):
    """All weights zero under "mean" divides by zero: the rows' gradients stay zero, also where
    the gradient that comes in is infinite or NaN."""
    d = make(4, V, 9, torch.float32, seed=18, holes=False)
    d["weights"][1] = d["weights"][2] = 0.0
    kw = dict(labels=d["labels"], weights=d["weights"], temperature=2.0, label_weight=0.3)
    args = (d["logits"], d["values"], d["indices"])
    lse = native.distill_forward(*args, **kw)["lse"]
    up = torch.tensor([1.0, float("inf"), float("nan"), float("nan")], device=DEV)
    g = native.distill_backward(*args, lse, up, **kw)
    assert not g[1:3].any() and bool(g[0].isfinite().all()) and bool(g[3].isnan().any())


@pytest.mark.parametrize("V", [1000, 5000])
@pytest.mark.parametrize("tau,lam", [(1.0, 0.0), (1.0, 0.4), (2.0, 0.5), (4.0, 0.3), (1.5, 0.5),
                                     (3.0, 0.0), (1.0, 1.0)])
def test_logits_far_from_zero(tau, lam, V):
    """A common offset of the logits drops out of the softmax: loss and gradient are as exact with
    it as without.  The backward takes log-sum-exps of up to 1024 as they are, rounded to 2^-24 of
    their size, and their products with 1/tau by half as much."""
    for offset in (300.0, 1e4, -3e5):
        d = make(7, V, 16, torch.float32, seed=19, holes=False)
        d["logits"] += offset
        ref, grad, size = reference(d, tau, lam)
        kw = dict(labels=d["labels"], weights=d["weights"], temperature=tau, label_weight=lam)
        args = (d["logits"], d["values"], d["indices"])
        s = native.distill_step(*args, **kw)
        f = native.distill_forward(*args, **kw)
        # a log-probability is a difference of at most 30 (a rounding or two of it, 4e-6) and a
        # logarithm that is off by 3e-5 at most; so is the loss, which averages them
        tol = d["weights"].double().cpu() * ((1 - lam) * tau ** 2 + lam) * 6e-5
        for got in (s["loss"], f["loss"]):
            assert bool(((got.double().cpu() - ref).abs() <= tol).all())
        check_grad(s["dlogits"], grad, size, torch.float32)
        got = native.distill_backward(*args, f["lse"], **kw)
        check_grad(got, grad, size * (1 + 1.5 * 1024 * 2.0 ** -24 / EPS), torch.float32)


@pytest.mark.parametrize("V", [300, 3001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_rows_of_extreme_logits(dtype, V):
    """Rows that a mask has filled with the type's lowest value, or with one far from zero, are
    uniform; beside one logit above the rest they are a point."""
    for tau, lam in ((1.0, 0.0), (1.0, 0.5), (2.0, 0.5), (4.0, 0.5), (1.5, 0.5), (3.0, 0.0), (0.5, 1.0)):
        d = make(6, V, 8, dtype, seed=21, holes=False)
        x = d["logits"]
        x[0], x[1], x[2], x[3] = torch.finfo(dtype).min, -1e9, torch.finfo(dtype).max, 3e10
        x[4] = torch.finfo(dtype).min
        x[4, 7] = 1.0
        d["indices"][4], d["labels"][4] = 7, 7       # else its loss is infinite
        ref, grad, size = reference(d, tau, lam)
        kw = dict(labels=d["labels"], weights=d["weights"], temperature=tau, label_weight=lam)
        args = (x, d["values"], d["indices"])
        s = native.distill_step(*args, **kw)
        f = native.distill_forward(*args, **kw)
        b = native.distill_backward(*args, f["lse"], **kw)
        tol = d["weights"].double().cpu() * ((1 - lam) * tau ** 2 + lam) * 6e-5
        assert bool(((s["loss"].double().cpu() - ref).abs() <= tol).all())
        assert torch.equal(s["loss"], f["loss"])
        # entries of row 4 lie on one column, whose share is their sum
        check_grad(s["dlogits"], grad, 2 * size, dtype)
        check_grad(b, grad, 2 * size, dtype)


@pytest.mark.parametrize("tau", [0.05, 100.0, 1000.0])
def test_extreme_temperatures(tau):
    for V in (900, 4001):
        d = make(6, V, 8, torch.float32, seed=22, holes=False)
        ref, grad, size = reference(d, tau, 0.3)
        kw = dict(labels=d["labels"], weights=d["weights"], temperature=tau, label_weight=0.3)
        args = (d["logits"], d["values"], d["indices"])
        s = native.distill_step(*args, **kw)
        # exponents of up to (range of 40) / tau carry two roundings of their size; the rest as in
        # the file's head
        eps = EPS + 2 * max(1.0, 40 / tau) * 2.0 ** -24
        check_grad(s["dlogits"], grad, size * eps / EPS, torch.float32)
        lse = native.distill_forward(*args, **kw)["lse"]
        eps += 1.5 * 1024 * 2.0 ** -24
        check_grad(native.distill_backward(*args, lse, **kw), grad, size * eps / EPS, torch.float32)


def test_logits_of_any_layout():
    """Transposed and broadcast logits, as any strided tensor of another operand."""
    d = make(6, 257, 8, torch.float32, seed=20, holes=False)
    args = (d["values"], d["indices"], d["labels"], d["weights"])
    kw = dict(temperature=2.0, label_weight=0.3, reduction="sum")
    z = d["logits"].clone().requires_grad_(True)
    (want,) = torch.autograd.grad(kfs.distill_loss(z, *args, **kw), z)
    t = d["logits"].t().contiguous().requires_grad_(True)
    (got,) = torch.autograd.grad(kfs.distill_loss(t.t(), *args, **kw), t)
    assert torch.equal(got.t(), want)
    one = d["logits"][:1].clone().requires_grad_(True)
    rows = d["logits"][:1].expand(6, 257).contiguous().requires_grad_(True)
    (want,) = torch.autograd.grad(kfs.distill_loss(rows, *args, **kw), rows)
    (got,) = torch.autograd.grad(kfs.distill_loss(one.expand(6, 257), *args, **kw), one)
    # the broadcast's gradient is the sum of six rows
    assert float((got - want.sum(0, keepdim=True)).abs().max()) <= 8 * 2.0 ** -24 * float(
        want.abs().sum(0).max())
