"""GPU tests of the gated Kronecker feed-forward half (kron_glu_forward / _backward through the
binding) against its definition in 64 bits (glu_reference.py).

BF16: every value within the bound that its roundings allow.  Outputs of 4096 values or more
also have a 2-norm of errors: a rounding to BF16 is a uniform error below 2^-8 of the value,
2^-8 / sqrt(3) in the mean square, and a value has at most eight of them behind it (C and T of
gate and of up, d, V, C again, the output), the gate's two times the activation's condition
number, at most 1.4 in the mean square over these inputs: sqrt(6 + 2 * 1.96) 2^-8 / sqrt(3) =
7.1e-3 for sums of terms of random sign.  8e-3 leaves a tenth for the sample.  Exact FP32:
1e-5 of the largest value, as for the layer."""
import ctypes
import math
import threading

import pytest
import torch

import kronecker_factored_structured_b200 as kfs
from glu_reference import reference
from kronecker_factored_structured_b200 import native

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
ACTS = ("silu", "gelu", "gelu_tanh", "sigmoid")


def make(N, p, q, m1, m2, r, dtype="bf16", seed=0, bias=True, zeros=0.3):
    g = torch.Generator().manual_seed(seed)
    t = native.io_dtype(dtype)
    S = torch.randn(2, p, q, generator=g) * 0.3 + 1
    S[torch.rand(2, p, q, generator=g) < zeros] = 0
    d = {"x": torch.randn(N, p * m1, generator=g), "S": S,
         "A": torch.randn(2, r, p, q, generator=g) / math.sqrt(p),
         "B": torch.randn(2, r, m1, m2, generator=g) / math.sqrt(m1),
         "dH": torch.randn(N, q * m2, generator=g)}
    if bias:
        d["bias"] = 0.3 * torch.randn(2, q * m2, generator=g)
    return {k: v.to(t).to(DEV) for k, v in d.items()}


def run(d, name, dtype):
    fac = (d["x"], d["S"], d["A"], d["B"])
    out = {"h": native.glu_forward(*fac, d.get("bias"), activation=name, dtype=dtype)}
    out.update(native.glu_backward(*fac, d["dH"], d.get("bias"), activation=name, dtype=dtype,
                                   need_dbias="bias" in d))
    native.device_error()
    return out


def compare(out, ref, dtype):
    for k, (v, bound) in ref.items():
        if out[k] is None:
            continue
        got = out[k].double()
        assert out[k].dtype == native.io_dtype(dtype) and got.shape == v.shape, k
        err = (got - v).abs()
        if dtype == "bf16":
            assert (err <= bound + 1e-30).all(), (k, float((err - bound).max()))
            norm = float(v.norm())
            if v.numel() >= 4096:
                assert float(err.norm()) <= 8e-3 * norm, (k, float(err.norm()) / norm)
        else:
            assert float(err.max()) <= 1e-5 * float(v.abs().max()) + 1e-30, k


# p, q, m1, m2, r: square, ragged groups, k slices (m2 > one MP), odd ranks, K chunks of x
# (m1 > 64), one group, many groups, blocks of 8, ranks that fill no block
SHAPES = [(4, 4, 16, 16, 1), (32, 32, 32, 32, 4), (24, 32, 32, 64, 1), (9, 11, 24, 40, 3),
          (1, 1, 8, 8, 1), (1, 17, 8, 8, 2), (17, 1, 40, 56, 5), (33, 35, 48, 24, 5),
          (64, 64, 64, 64, 8), (5, 6, 72, 8, 1), (6, 5, 8, 72, 2), (3, 4, 128, 128, 3),
          (128, 40, 8, 16, 1), (40, 128, 16, 8, 2), (8, 200, 16, 16, 1), (13, 7, 136, 104, 1),
          (64, 8, 16, 64, 7), (2, 300, 8, 8, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "p{}q{}_m{}x{}_r{}".format(*s))
def test_bf16_shapes(shape):
    for N in (1, 37, 300):
        name = ACTS[(N + shape[0]) % 4]
        d = make(N, *shape, seed=N, bias=N != 37)
        compare(run(d, name, "bf16"), reference(d, name), "bf16")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("N", [2, 3, 4, 5, 8, 9, 16, 129, 2111])
def test_bf16_rows(N, name):
    d = make(N, 12, 20, 32, 32, 2, seed=N)
    compare(run(d, name, "bf16"), reference(d, name), "bf16")


F32 = [(32, 32, 32, 32, 4, 2500), (128, 128, 8, 8, 2, 19), (64, 64, 64, 64, 2, 5),
       (4, 4, 4, 4, 1, 3), (9, 11, 12, 20, 3, 37), (32, 32, 32, 32, 4, 65), (1, 1, 4, 4, 1, 1),
       (32, 24, 16, 32, 2, 777), (7, 3, 28, 8, 2, 150)]


@pytest.mark.parametrize("case", F32, ids=lambda s: "p{}q{}_m{}x{}_r{}_N{}".format(*s))
def test_f32(case):
    *shape, N = case
    for k, name in enumerate(ACTS):
        d = make(N, *shape, dtype="f32", seed=k, bias=k != 1)
        compare(run(d, name, "f32"), reference(d, name), "f32")


# several passes over the ranks, the last one shorter; several tiles per CTA in each form; a last
# slice of k that is narrower; more columns c than one kernel takes; a backward in tiles of one and
# of several slots, the last tile shorter, and in one that does not fit
F32_TILES = [(30, 30, 32, 32, 4, 300), (5, 7, 4, 12, 1, 1000), (4, 36, 20, 8, 2, 149),
             (48, 48, 24, 24, 1, 2000), (32, 32, 32, 32, 9, 300),
             (64, 64, 32, 32, 6, 2000), (8, 8, 12, 20, 3, 6000),
             (40, 33, 28, 44, 5, 1200), (3, 70, 8, 100, 2, 33), (2, 2100, 4, 4, 1, 5)]


@pytest.mark.parametrize("case", F32_TILES, ids=lambda s: "p{}q{}_m{}x{}_r{}_N{}".format(*s))
def test_f32_passes_and_tiles(case):
    *shape, N = case
    d = make(N, *shape, dtype="f32", seed=N)
    name = ACTS[N % 4]
    compare(run(d, name, "f32"), reference(d, name), "f32")


def test_many_rows():
    """More tiles than CTAs, several row ranges of the weight gradient, a ragged last tile."""
    d = make(20003, 16, 16, 16, 32, 2, seed=9)
    compare(run(d, "silu", "bf16"), reference(d, "silu"), "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_batch(dtype):
    d = make(0, 4, 4, 16, 16, 2, dtype=dtype)
    fac = (d["x"], d["S"], d["A"], d["B"])
    assert native.glu_forward(*fac, d["bias"], dtype=dtype).shape == (0, 64)
    filled = {k: torch.full(s, 7.0, device=DEV, dtype=native.io_dtype(dtype))
              for k, s in (("dS", (2, 4, 4)), ("dA", (2, 2, 4, 4)), ("dB", (2, 2, 16, 16)),
                           ("dbias", (2, 64)))}
    g = native.glu_backward(*fac, d["dH"], d["bias"], dtype=dtype, grads=filled)
    assert all(not g[k].any() for k in filled)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_not_asked_for(dtype):
    d = make(50, 6, 5, 16, 24, 2, dtype=dtype)
    fac = (d["x"], d["S"], d["A"], d["B"], d["dH"], d["bias"])
    full = native.glu_backward(*fac, dtype=dtype)
    part = native.glu_backward(*fac, dtype=dtype, need_dx=False, need_dbias=False)
    assert part["dX"] is None and part["dbias"] is None
    for k in ("dS", "dA", "dB"):
        assert torch.equal(full[k], part[k])


def test_memory_behind_the_last_row_stays():
    N = 37
    d = make(N, 9, 11, 24, 40, 3)
    h = torch.full((N + 8, 440), 7.0, dtype=torch.bfloat16, device=DEV)
    dx = torch.full((N + 8, 216), 7.0, dtype=torch.bfloat16, device=DEV)
    fac = (d["x"], d["S"], d["A"], d["B"])
    native.glu_forward(*fac, d["bias"], out=h[:N])
    native.glu_backward(*fac, d["dH"], d["bias"], grads={"dX": dx[:N]})
    assert bool((h[N:] == 7).all()) and bool((dx[N:] == 7).all())
    assert not bool((h[:N] == 7).all())


def test_a_nan_stays_in_its_row():
    d = make(21, 9, 11, 24, 40, 3)
    clean = run(d, "silu", "bf16")
    d["x"][5, 3] = float("nan")
    d["dH"][9, 7] = float("inf")
    bad = run(d, "silu", "bf16")
    rows = torch.arange(21, device=DEV) != 5
    assert torch.equal(bad["h"][rows], clean["h"][rows]) and bool(bad["h"][5].isnan().any())
    rows &= torch.arange(21, device=DEV) != 9
    assert torch.equal(bad["dX"][rows], clean["dX"][rows])


def test_saturated_activations():
    """Pre-activations of some hundreds: the exponentials overflow and vanish."""
    for name in ACTS:
        for dtype in ("f32", "bf16"):
            d = make(33, 8, 8, 16, 16, 2, dtype=dtype, zeros=0.0)
            d["x"] *= 200
            out, ref = run(d, name, dtype), reference(d, name)
            assert all(bool(out[k].isfinite().all()) for k in out)
            if dtype == "f32":
                assert float((out["h"].double() - ref["h"][0]).abs().max()) <= 1e-5 * float(
                    ref["h"][0].abs().max())


def test_gradients_against_differences():
    d = make(5, 3, 4, 8, 12, 2, dtype="f32")
    g = run(d, "gelu", "f32")
    eps = 2.0 ** -6
    gen = torch.Generator().manual_seed(1)
    for key, grad in (("x", "dX"), ("S", "dS"), ("A", "dA"), ("B", "dB"), ("bias", "dbias")):
        v = torch.randn(d[key].shape, generator=gen).to(DEV)
        v /= v.norm()
        f = []
        for s in (-eps, eps):
            e = dict(d)
            e[key] = d[key] + s * v
            h = native.glu_forward(e["x"], e["S"], e["A"], e["B"], e["bias"], "gelu", "f32")
            f.append(float((h.double() * d["dH"].double()).sum()))
        got, scale = float((g[grad].double() * v.double()).sum()), float(g[grad].norm())
        # eps^2 / 6 times a third derivative of a few times the gradient, and 1e-6 / eps of
        # rounding in f
        assert abs((f[1] - f[0]) / (2 * eps) - got) <= 2e-3 * (1 + scale)


def test_stream_graph_and_repeat():
    d = make(513, 24, 32, 32, 64, 2, seed=3)
    want = run(d, "silu", "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = run(d, "silu", "bf16")
    b = run(d, "silu", "bf16")
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(a[k], want[k]) and torch.equal(b[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    fac = (d["x"], d["S"], d["A"], d["B"])
    with torch.cuda.graph(graph):
        h = native.glu_forward(*fac, d["bias"])
        g = native.glu_backward(*fac, d["dH"], d["bias"])
    other = make(513, 24, 32, 32, 64, 2, seed=4)
    for k in d:
        d[k].copy_(other[k])
    graph.replay()
    torch.cuda.synchronize()
    fresh = run(d, "silu", "bf16")
    assert torch.equal(h, fresh["h"])
    for k in g:
        assert torch.equal(g[k], fresh[k]), k


@pytest.mark.parametrize("shape", [(30, 22, 12, 20, 2), (32, 32, 32, 32, 9)],
                         ids=["one_pass", "several_passes"])
def test_f32_nan_row_graph_and_last_row(shape):
    N, (p, q, m1, m2, r) = 213, shape
    d = make(N, *shape, dtype="f32", seed=3)
    clean = run(d, "silu", "f32")
    bad = {k: v.clone() for k, v in d.items()}
    bad["x"][5, 3], bad["dH"][9, 7] = float("nan"), float("inf")
    got = run(bad, "silu", "f32")
    rows = torch.arange(N, device=DEV) != 5
    assert torch.equal(got["h"][rows], clean["h"][rows]) and bool(got["h"][5].isnan().any())
    rows &= torch.arange(N, device=DEV) != 9
    assert torch.equal(got["dX"][rows], clean["dX"][rows])

    fac = (d["x"], d["S"], d["A"], d["B"])
    h = torch.full((N + 7, q * m2), 7.0, device=DEV)
    grads = {"dX": torch.full((N + 7, p * m1), 7.0, device=DEV)[:N]}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.glu_forward(*fac, d["bias"], dtype="f32", out=h[:N])
        g = native.glu_backward(*fac, d["dH"], d["bias"], dtype="f32", grads=grads)
    other = make(N, *shape, dtype="f32", seed=4)
    for k in d:
        d[k].copy_(other[k])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    fresh = run(d, "silu", "f32")
    assert torch.equal(h[:N], fresh["h"]) and bool((h[N:] == 7).all())
    for k in g:
        assert torch.equal(g[k], fresh[k]), k
    behind = torch.as_strided(grads["dX"], (7, p * m1), (p * m1, 1), N * p * m1)
    assert bool((behind == 7).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_module_and_autograd(dtype):
    torch.manual_seed(0)
    glu = kfs.KronGLU(96, 160, 16, 32, rank=2, activation="gelu_tanh", dtype=dtype, device=DEV)
    with torch.no_grad():
        glu.bias.normal_(0, 0.2)
    t = native.io_dtype(dtype)
    x = torch.randn(3, 7, 96, device=DEV).to(t).requires_grad_(True)
    up = torch.randn(3, 7, 160, device=DEV).to(t)
    h = glu(x)
    assert h.shape == (3, 7, 160)
    h.backward(up)
    d = {"x": x.detach().reshape(21, 96), "S": glu.S.detach(), "A": glu.A.detach(),
         "B": glu.B.detach(), "bias": glu.bias.detach(), "dH": up.reshape(21, 160)}
    out = {"h": h.detach().reshape(21, 160), "dX": x.grad.reshape(21, 96), "dS": glu.S.grad,
           "dA": glu.A.grad, "dB": glu.B.grad, "dbias": glu.bias.grad}
    compare(out, reference(d, "gelu_tanh"), dtype)


def test_gated_block_distilled_on_its_teachers_top_logits():
    """The operators together, as a compressed block is trained: gated half, down projection,
    head, loss against the top logits of a dense teacher, all gradients, and a captured step
    that repeats the eager one."""
    torch.manual_seed(1)
    ffn = kfs.KronGatedFFN(256, 256, 32, rank=2, dtype="f32", device=DEV)
    head = torch.nn.Linear(256, 1003, device=DEV)
    x = torch.randn(4, 33, 256, device=DEV)
    with torch.no_grad():
        values, indices = (3 * torch.randn(4, 33, 1003, device=DEV)).topk(20)
    loss_fn = kfs.DistillLoss(temperature=2.0)
    params = list(ffn.parameters()) + list(head.parameters())

    def step():
        return torch.autograd.grad(loss_fn(head(ffn(x)), values, indices), params)

    got = step()
    y = x.double()
    glu, down = ffn.glu, ffn.down
    ps = [p.detach().double().requires_grad_(True) for p in params]
    it = iter(ps)
    S, A, B, b, Sd, Ad, Bd, bd, Wh, bh = it
    dense = lambda S, A, B: sum(torch.kron(S * A[i], B[i]) for i in range(A.shape[0]))  # noqa: E731
    assert [p.shape for p in params[:4]] == [glu.S.shape, glu.A.shape, glu.B.shape, glu.bias.shape]
    assert params[4] is down.S
    g = y @ dense(S[0], A[0], B[0]) + b[0]
    u = y @ dense(S[1], A[1], B[1]) + b[1]
    z = (g * torch.sigmoid(g) * u) @ dense(Sd, Ad, Bd) + bd
    z = z @ Wh.t() + bh
    p = torch.softmax(values.double() / 2, -1)
    logq = torch.log_softmax(z / 2, -1).gather(-1, indices)
    loss = 4 * (p * (p.log() - logq)).sum(-1).mean()
    want = torch.autograd.grad(loss, ps)
    for a, w in zip(got, want):
        # fp32 throughout: 1e-5 of the largest value per operator, four in a row
        assert float((a.double() - w).abs().max()) <= 4e-5 * float(w.abs().max())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, w in zip(again[:8], got[:8]):
        assert torch.equal(a, w)


def test_offsets_beyond_32_bits():
    """2,097,161 rows of 1024: element offsets pass 2^31 in x, h, dH and dX.  Rows are
    independent, so the last ones are checked."""
    N, shape = (1 << 21) + 9, (32, 32, 32, 32, 1)
    d = make(64, *shape, seed=21)
    x = torch.zeros(N, 1024, dtype=torch.bfloat16, device=DEV)
    dH = torch.zeros(N, 1024, dtype=torch.bfloat16, device=DEV)
    x[-64:], dH[-64:] = d["x"], d["dH"]
    fac = (x, d["S"], d["A"], d["B"])
    h = native.glu_forward(*fac, d["bias"])
    g = native.glu_backward(*fac, dH, d["bias"])
    native.device_error()
    out = {"h": h[-64:], "dX": g["dX"][-64:], "dA": g["dA"], "dB": g["dB"], "dS": g["dS"],
           "dbias": g["dbias"]}       # the other rows' gradients are zero
    compare(out, reference(d, "silu"), "bf16")
    assert not g["dX"][:-64][:: 4097].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_streams_at_once(dtype):
    """Calls on streams of their own, given to the binding, with workspaces of their own."""
    ds = [make(700 + 13 * i, 16, 24, 16, 32, 2, dtype=dtype, seed=i) for i in range(3)]
    want = [run(d, "silu", dtype) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for d, s in zip(ds, streams):
            fac = (d["x"], d["S"], d["A"], d["B"])
            g = native.glu_backward(*fac, d["dH"], d["bias"], dtype=dtype, stream=s)
            g["h"] = native.glu_forward(*fac, d["bias"], dtype=dtype, stream=s)
            got.append(g)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(g[k], w[k]) for k in w)


def test_given_workspace_and_outputs():
    d = make(300, 9, 11, 24, 40, 3)
    fac = (d["x"], d["S"], d["A"], d["B"])
    n = native.glu_workspace_size(300, 9, 11, 24, 40, 3, "bf16", True)
    ws = torch.full((n + 512,), 0x7F, dtype=torch.uint8, device=DEV)      # NaN everywhere
    guard = ws[n:].clone()
    g = native.glu_backward(*fac, d["dH"], d["bias"], workspace=ws[:n])
    assert torch.equal(ws[n:], guard)
    for k, v in native.glu_backward(*fac, d["dH"], d["bias"]).items():
        assert torch.equal(v, g[k]), k
    with pytest.raises(native.KronError):
        native.glu_backward(*fac, d["dH"], d["bias"], workspace=ws[: n - 256])
    # dX over dH
    sq = make(77, 8, 8, 16, 16, 2)
    fac = (sq["x"], sq["S"], sq["A"], sq["B"])
    want = native.glu_backward(*fac, sq["dH"], sq["bias"])
    got = native.glu_backward(*fac, dh := sq["dH"].clone(), sq["bias"], grads={"dX": dh})
    assert all(torch.equal(want[k], got[k]) for k in want)
    with pytest.raises(native.KronError):
        native.glu_backward(*fac, sq["dH"], sq["bias"], grads={"dX": sq["x"]})
    with pytest.raises(native.KronError):
        native.glu_forward(*fac, sq["bias"], out=sq["x"])


def _tails(g, name):
    """act(g), act'(g) and the terms that act' is the sum of, in absolute value; in 64 bits, in
    forms that do not cancel (1 + tanh(v) = 2 sigmoid(2 v), 1 + erf(v) = erfc(-v))."""
    if name == "gelu":
        c = torch.special.erfc(-g / math.sqrt(2)) / 2
        slope = g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        return g * c, c + slope, c + slope.abs(), 1 + g.abs()
    v, dv = g, torch.ones_like(g)
    if name == "gelu_tanh":
        v = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
        dv = math.sqrt(8 / math.pi) * (1 + 0.134145 * g ** 2)
    s, c = torch.sigmoid(v), torch.sigmoid(-v)
    if name == "sigmoid":
        return s, s * c, s * c, 1 + 0 * g
    return g * s, s + g * dv * s * c, s + (g * dv).abs() * s * c, 1 + (g * dv).abs()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ACTS)
def test_tails_of_the_activations(name, dtype):
    """x = 0, so the bias is the pre-activation: the activation and its derivative alone, to
    their own size.  f32: 2^-20 for the functions, and exponents of up to 150 rounded once or
    twice (2 * 150 * 2^-24 < 2^-15 of an exponential); bf16: 2^-8 besides, for the rounding of
    what is stored.  An exponential of 2^126 or more may be infinite, so that what it divides is
    zero: 2^-126 of the factors that it has."""
    g = torch.arange(-96, 161, dtype=torch.float64).div(8)            # -12 to 20
    d = make(1, 2, 33, 8, 8, 1, dtype=dtype)
    bias = torch.ones(2, 264, dtype=torch.float64)
    bias[0, : g.numel()] = g
    g = bias[0]
    d["x"].zero_()
    d["dH"].fill_(1.0)
    d["bias"] = bias.to(native.io_dtype(dtype)).to(DEV)
    assert torch.equal(d["bias"].double().cpu(), bias)                # nothing is rounded
    out = run(d, name, dtype)
    f, df, terms, factor = _tails(g, name)
    fn = 2.0 ** -15 + 2.0 ** -20
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    low = 2.0 ** -126 * factor
    err = (out["h"][0].double().cpu() - f).abs()
    assert bool((err <= (fn + half) * f.abs() + low).all()), g[err > (fn + half) * f.abs() + low]
    # of one row: the column sum is dg itself
    err, tol = (out["dbias"][0].double().cpu() - df).abs(), fn * terms + half * df.abs() + low
    assert bool((err <= tol).all()), g[err > tol]


# dtype, and two sizes (N, p, q, m1, m2, r) that run the same instantiations of the kernels with
# tiles of different size: the kernels on the tensor cores, the factor gradients of few rows, the
# exact-FP32 kernels, and the layer's FP32 backward beside a gated one that runs its kernel
THREADS = [("bf16", (300, 32, 32, 32, 32, 4), (300, 2, 2, 32, 32, 1)),
           ("bf16", (8, 300, 2, 8, 8, 1), (8, 4, 4, 8, 8, 1)),
           ("f32", (37, 30, 22, 12, 20, 2), (5, 2, 2, 4, 4, 1)),
           ("f32", (9, 4, 4, 64, 64, 8), (5, 2, 2, 8, 8, 1))]


@pytest.mark.parametrize("case", range(4), ids=["bf16", "bf16_few_rows", "f32", "f32_layer"])
def test_host_threads_at_once(case):
    """Calls of two sizes from several host threads, which meet inside the library: every one
    succeeds, and gives what it gives alone."""
    dtype, *sizes = THREADS[case]
    lib = native.load()

    def setup(k):
        N, *shape = sizes[k]
        d = make(N, *shape, dtype=dtype, seed=k)
        fac = [d[n] for n in ("x", "S", "A", "B")]
        stream = torch.cuda.Stream()
        p, q, m1, m2, r = shape
        tail = (N, p, q, m1, m2, r)
        if case == 3 and k == 1:      # the layer
            fac[1:] = [t[0].contiguous() for t in fac[1:]]
            want = kfs.backward(*fac, d["dH"], dtype=dtype)
            n = kfs.workspace_size(*tail, dtype)
        else:
            want = native.glu_backward(*fac, d["dH"], d["bias"], dtype=dtype)
            want["h"] = native.glu_forward(*fac, d["bias"], dtype=dtype)
            n = native.glu_workspace_size(*tail, dtype, True)
        out = {n: torch.zeros_like(v) for n, v in want.items()}
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
        P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        fp = [P(t) for t in fac]
        grads = [P(out[n]) for n in ("dX", "dS", "dA", "dB", "dbias")]
        end = (native.DTYPES[dtype], 0, P(ws), ws.numel(), ctypes.c_void_p(stream.cuda_stream))
        if case == 3 and k == 1:
            calls = [(lib.kron_linear_backward, (*fp, P(d["dH"]), *grads, *tail, *end))]
        else:
            bias = P(d["bias"])
            calls = [(lib.kron_glu_forward, (*fp, bias, P(out["h"]), *tail, 0, *end)),
                     (lib.kron_glu_backward, (*fp, bias, P(d["dH"]), *grads, *tail, 0, *end))]
        return want, out, calls, stream, (d, fac, ws)

    work = [setup(k) for k in (0, 1, 0, 1, 0, 1)]
    torch.cuda.synchronize()
    failed = []
    start = threading.Barrier(len(work))

    def loop(i):
        _, _, calls, stream, _ = work[i]
        start.wait()
        for n in range(2000):
            for f, args in calls:
                if f(*args):
                    failed.append(lib.kron_last_error().decode())
            if n % 100 == 99:
                stream.synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, (len(failed), failed[:3])
    for want, out, *_ in work:
        for n in want:
            assert torch.equal(out[n], want[n]), n


def test_forward_without_a_backward():
    """Sizes whose forward has a kernel and whose gradients have none."""
    for dtype, N, shape in (("bf16", 37, (64, 224, 64, 64, 8)), ("f32", 9, (128, 128, 64, 64, 1))):
        d = make(N, *shape, dtype=dtype, seed=5)
        fac = (d["x"], d["S"], d["A"], d["B"])
        ref = reference({k: v for k, v in d.items() if k != "dH"}, "silu")
        compare({"h": native.glu_forward(*fac, d["bias"], dtype=dtype)}, ref, dtype)
        with pytest.raises(native.KronError):
            native.glu_backward(*fac, d["dH"], d["bias"], dtype=dtype)
