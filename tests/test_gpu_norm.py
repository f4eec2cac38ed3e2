"""GPU tests of the group norm with an activation, channels last, and its gradient
against the formulas in 64 bits.

Tolerances, relative to the 2-norm of the tensor, before any run: fp32 results 1e-5
(sums of at most 2048 products, each partial sum off by 2^-24; the exponential of the
activation a few units in the last place); sums over rows the same (their terms are
summed in lines of a few hundred); bf16 results one rounding, at most 2^-8 of each
element.
"""
import numpy as np
import pytest
import torch

import linear_rnn_sequence_amd as dp
from parity import f64, say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    dp.load()


def sigmoid(a):
    return 1.0 / (1.0 + np.exp(-a))


def reference(x, w, b, z, dy, eps, rms, silu):
    m = 0.0 if rms else x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    n = (x - m) * r
    a = n * (1.0 if w is None else w) + (0.0 if b is None else b)
    g = {}
    if z is not None:
        s = sigmoid(z)
        y, da = a * z * s, dy * z * s
        g["gate"] = dy * a * (s + z * s * (1 - s))
    elif silu:
        s = sigmoid(a)
        y, da = a * s, dy * (s + a * s * (1 - s))
    else:
        y, da = a, dy
    lead = tuple(range(x.ndim - 2))
    if w is not None:
        g["weight"] = (da * n).sum(lead)
    if b is not None:
        g["bias"] = da.sum(lead)
    dn = da * (1.0 if w is None else w)
    d = dn - n * (dn * n).mean(-1, keepdims=True)
    if not rms:
        d = d - dn.mean(-1, keepdims=True)
    g["x"] = r * d
    return y, g, r * dn


def check(label, got, ref, low, terms=None):
    """terms: what the result is a difference of.  dx = r dn - r mean(dn) - r n mean(dn n)
    carries the fp32 rounding of terms as large as r dn, each off by 2^-24 of itself, so
    its fp32 error is held to r dn's size.  That differs from dx's own size where the
    terms cancel: in a group of two channels n = +-(1 - eps / (2 var)), and
    dx = r (dn - mean(dn)) (1 - n^2) is about eps / var = 1e-6 of each term."""
    got = f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), label
    norm = max(np.linalg.norm(ref), 0.0 if terms is None else np.linalg.norm(terms))
    rms = norm / np.sqrt(max(1, ref.size)) or 1.0
    err = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) if low else 0)
    rel = np.linalg.norm(got - ref) / norm if norm else np.linalg.norm(got - ref)
    say(f"  {label}: rel {rel:.2e}, worst element {err.max():.2e} / RMS {rms:.2e}")
    assert rel <= (2.0 ** -8 if low else 1e-5), label
    assert err.max() <= 4e-4 * rms, label


# leading sizes, G, D: one row, one channel, odd widths (no 16-byte vectors), each split
# of a group over lanes (4 .. 64 lanes, 1 .. 8 vectors), more groups than a workgroup holds
CASES = [
    ((1,), 1, 1), ((3,), 2, 2), ((7,), 5, 3), ((2, 9), 4, 16), ((33,), 70, 8), ((64,), 16, 64),
    ((2, 50), 16, 128), ((129,), 3, 100), ((40,), 12, 100), ((17,), 2, 255), ((1000,), 1, 256), ((9,), 5, 333),
    ((31,), 2, 768), ((5,), 3, 1000), ((4,), 1, 2047), ((6,), 2, 2048), ((3001,), 8, 24),
]
ACTS = ["none", "silu", "gate"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, (*c[0], c[1], c[2]))) for c in CASES])
def test_norm_and_gradient(case, dtype):
    lead, G, D = case
    gen = torch.Generator().manual_seed(G * 1000 + D)
    for i, act in enumerate(ACTS):
        rms, affine = (i + G + D) % 2 == 1, (i + D) % 3 != 0
        eps = 1e-5 if D > 1 else 0.1
        n = lambda *s: torch.randn(*s, generator=gen)
        x, dy = (n(*lead, G, D) * 3 + 1).to(DT[dtype]), n(*lead, G, D).to(DT[dtype])
        w, b = (1 + 0.2 * n(G, D), 0.2 * n(G, D)) if affine else (None, None)
        z = n(*lead, G, D).to(DT[dtype]) if act == "gate" else None
        say(f"case norm {case} {dtype} {act} rms={rms} affine={affine}")
        c = lambda t: None if t is None else t.cuda()
        y = dp.group_norm(c(x), c(w), c(b), c(z), eps=eps, rms=rms, silu=act == "silu")
        g = dp.group_norm_bwd(c(x), c(dy), c(w), c(b), c(z), eps=eps, rms=rms, silu=act == "silu")
        torch.cuda.synchronize()
        f = lambda t: None if t is None else f64(t)
        ry, rg, terms = reference(f64(x), f(w), f(b), f(z), f64(dy), eps, rms, act == "silu")
        low = dtype == "bf16"
        if D == 1 and not rms:  # x - mean is zero: the result is the bias, dx is zero
            assert float(g["x"].abs().max()) <= 1e-6
            rg.pop("x")
        check("y", y, ry, low)
        assert set(g) == set(rg) | {"x"}
        for k, r in rg.items():
            check(k, g[k], r, low and k in ("x", "gate"), terms if k == "x" else None)


def test_gradient_against_differences():
    gen = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    for act, rms in (("gate", False), ("silu", True), ("none", False)):
        t = dict(x=n(6, 3, 20), weight=1 + 0.2 * n(3, 20), bias=0.2 * n(3, 20), gate=n(6, 3, 20) if act == "gate" else None)
        t = {k: None if v is None else v.float().double() for k, v in t.items()}
        dy = n(6, 3, 20).float().double()
        c = lambda k: None if t[k] is None else t[k].float().cuda()
        g = dp.group_norm_bwd(c("x"), dy.float().cuda(), c("weight"), c("bias"), c("gate"), rms=rms, silu=act == "silu")

        def loss(d):
            a = [None if d[k] is None else d[k].numpy() for k in ("x", "weight", "bias", "gate")]
            return float((reference(*a, dy.numpy(), 1e-5, rms, act == "silu")[0] * dy.numpy()).sum())

        for k in g:
            u, e = n(*t[k].shape), 1e-5
            hi, lo = dict(t), dict(t)
            hi[k], lo[k] = t[k] + e * u, t[k] - e * u
            fd, an = (loss(hi) - loss(lo)) / (2 * e), float((f64(g[k]) * u.numpy()).sum())
            # rounding of g on a random direction, four standard deviations; the differences' e^2 and 1 / e errors
            assert abs(fd - an) <= (4e-5 + 1e-6) * np.linalg.norm(f64(g[k])) + 1e-6, (act, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_offsets_and_constant_rows(dtype):
    """A mean far above the spread (the variance is not a difference of sums), a constant
    row, and rows whose squares stay in range."""
    x = torch.randn(4, 2, 96, generator=torch.Generator().manual_seed(1))
    x[0] += 1000.0
    x[1] = 5.0
    x[2] *= 1e6
    x[3] *= 1e-6
    x = x.to(DT[dtype])
    y = dp.group_norm(x.cuda())
    ry, _, _ = reference(f64(x), None, None, None, np.zeros(x.shape), 1e-5, False, False)
    assert bool((y[1] == 0).all())
    for r in (0, 2, 3):
        # at 1000 the fp32 mean of 96 values is off by a few 2^-24 * 1000 = 6e-5 each
        np.testing.assert_allclose(f64(y[r]), ry[r], atol=2e-4, rtol=2.0 ** -8 if dtype == "bf16" else 1e-5)


@pytest.mark.parametrize("rms", [False, True])
def test_tiny_spreads_without_eps(rms):
    """Mean squares around the smallest normal float: of values 2^-61 .. 2^-67 they are
    2^-122 .. 2^-134, the smaller ones denormal with 2^-149 as their step.  Each of the 64
    squares is off by half a step at most, so is their mean (2^-150 from either) of m2 >=
    2^-135, which is 2^-14 of m2 and 2^-15 of n, |n| < 2; the mean of x is off by a few 2^-24
    of the largest value."""
    for e in (-61, -64, -67):
        x = torch.randn(6, 3, 64, generator=torch.Generator().manual_seed(4)).sign() * 2.0 ** e
        x[:, :, ::5] *= 0.5
        y = dp.group_norm(x.cuda(), eps=0.0, rms=rms).cpu().double()
        X = x.double() - (0 if rms else x.double().mean(-1, keepdim=True))
        want = X / (X * X).mean(-1, keepdim=True).sqrt()
        assert float((y - want).abs().max()) <= 2.0 ** -15 * 2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("D", [3, 64, 100, 2048])
def test_large_values(D, rms, dtype):
    """Rows whose squares (1e25) and whose sums (3e37 and an offset of 1e38) pass fp32's range
    beside ordinary ones: the result has none of their size, and the gradient is 1 / spread of
    it.  The mean of values on an offset is off by a few 2^-24 of the offset, here 3 times the
    spread, and so is taken out: as in any row."""
    gen = torch.Generator().manual_seed(D)
    n = lambda *s: torch.randn(*s, generator=gen).clamp(-3, 3)
    x, dy = n(6, 2, D), n(6, 2, D)
    x[1] *= 1e25
    x[3] = x[3] * 3e37 + (0 if rms else 1e38)
    x[4] *= 1e19
    x, dy = x.to(DT[dtype]), dy.to(DT[dtype])
    y = dp.group_norm(x.cuda(), rms=rms)
    g = dp.group_norm_bwd(x.cuda(), dy.cuda(), rms=rms)
    torch.cuda.synchronize()
    ry, rg, terms = reference(f64(x), None, None, None, f64(dy), 1e-5, rms, False)
    for i in range(6):  # row by row: their gradients are of different sizes
        check(f"y {i}", y[i], ry[i], dtype == "bf16")
        if i != 3:  # 1 / 3e37 is a denormal's size
            check(f"x {i}", g["x"][i], rg["x"][i], dtype == "bf16", terms[i])


def test_large_values_and_eps():
    """An eps next to squares past fp32's range (2^128) counts as next to smaller ones."""
    x = torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(5)) * 3e19
    y = dp.group_norm(x.cuda(), eps=1e38)
    check("y", y, reference(f64(x), None, None, None, np.zeros(x.shape), 1e38, False, False)[0], False)


def test_saturated_gates():
    z = torch.tensor([-200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 1e30]).repeat(2).reshape(1, 1, 16)
    x = torch.arange(16.0).reshape(1, 1, 16)
    y = dp.group_norm(x.cuda(), gate=z.cuda())
    g = dp.group_norm_bwd(x.cuda(), torch.ones(1, 1, 16).cuda(), gate=z.cuda())
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(g["gate"]).all())


def test_in_place_streams_replays_and_empty():
    gen = torch.Generator().manual_seed(2)
    x, z, dy = (torch.randn(300, 4, 128, generator=gen).bfloat16().cuda() for _ in range(3))
    w, b = torch.rand(4, 128, generator=gen).cuda(), torch.rand(4, 128, generator=gen).cuda()
    y, g = dp.group_norm(x, w, b, z), dp.group_norm_bwd(x, dy, w, b, z)
    g2 = dp.group_norm_bwd(x, dy, w, b, z)
    assert all(torch.equal(g[k], g2[k]) for k in g)
    xi = x.clone()
    assert dp.group_norm(xi, w, b, z, out=xi) is xi and torch.equal(xi, y)
    dyi, zi = dy.clone(), z.clone()
    gi = dp.group_norm_bwd(x, dyi, w, b, zi, grads=dict(x=dyi, gate=zi))
    assert all(torch.equal(g[k], gi[k]) for k in g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gs = dp.group_norm_bwd(x, dy, w, b, z, stream=side)
    side.synchronize()
    assert all(torch.equal(g[k], gs[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cy, cg = dp.group_norm(x, w, b, z), dp.group_norm_bwd(x, dy, w, b, z)
    for i in range(4):
        x.copy_(torch.randn(300, 4, 128, generator=gen).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        y, g = dp.group_norm(x, w, b, z), dp.group_norm_bwd(x, dy, w, b, z)
        assert torch.equal(cy, y) and all(torch.equal(cg[k], g[k]) for k in g)
    e = torch.empty(0, 4, 128, device="cuda")
    assert dp.group_norm(e, w, b).shape == e.shape
    g = dp.group_norm_bwd(e, e, w, b)
    assert g["x"].shape == e.shape and bool((g["weight"] == 0).all()) and bool((g["bias"] == 0).all())


def test_gradients_left_out():
    gen = torch.Generator().manual_seed(8)
    x, z, dy = (torch.randn(50, 4, 64, generator=gen).cuda() for _ in range(3))
    w, b = torch.rand(4, 64, generator=gen).cuda(), torch.rand(4, 64, generator=gen).cuda()
    g = dp.group_norm_bwd(x, dy, w, b, z)
    for left in (["weight"], ["bias"], ["weight", "bias"]):
        part = dp.group_norm_bwd(x, dy, w, b, z, grads={n: None for n in left})
        assert all(part[n] is None if n in left else torch.equal(g[n], part[n]) for n in g)
    with pytest.raises(dp.DPError):
        dp.group_norm_bwd(x, dy, w, b, z, grads=dict(x=None))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G,D", [(5, 1), (3, 3), (7, 33), (12, 100), (2, 2047)])
def test_in_place_at_odd_widths(G, D, dtype):
    """y over x, dx over dy and the gate's gradient over the gate, where a group's last vector
    is read from its neighbour channels and written by parts: the bits of separate buffers."""
    gen = torch.Generator().manual_seed(D)
    x, z, dy = (torch.randn(41, G, D, generator=gen).to(DT[dtype]).cuda() for _ in range(3))
    w, b = torch.rand(G, D, generator=gen).cuda(), torch.rand(G, D, generator=gen).cuda()
    for gate in (z, None):
        y, g = dp.group_norm(x, w, b, gate, silu=gate is None), dp.group_norm_bwd(x, dy, w, b, gate, silu=gate is None)
        xi, dyi, zi = x.clone(), dy.clone(), None if gate is None else gate.clone()
        gi = dp.group_norm_bwd(x, dyi, w, b, zi, silu=gate is None, grads=dict(x=dyi) if gate is None else dict(x=dyi, gate=zi))
        assert dp.group_norm(xi, w, b, gate, silu=gate is None, out=xi) is xi and torch.equal(xi, y)
        assert set(gi) == set(g) and all(torch.equal(g[k], gi[k]) for k in g)


def test_layer_linear_attention_norm_gate():
    """Linear attention, its norm with a SiLU gate, and the gradient through both, as a
    layer runs them, against fp64 autograd of the definition."""
    B, L, H, Hk, dk, dv = 1, 150, 4, 2, 64, 64
    gen = torch.Generator().manual_seed(6)
    n = lambda *s: torch.randn(*s, generator=gen)
    t = dict(q=n(B, L, Hk, dk) * dk ** -0.5, k=n(B, L, Hk, dk), v=n(B, L, H, dv), ld=-torch.rand(B, L, H, generator=gen) * 0.3,
             w=1 + 0.1 * n(H, dv), b=0.1 * n(H, dv), z=n(B, L, H, dv))
    dy = n(B, L, H, dv)
    c = {k: v.cuda() for k, v in t.items()}
    o, _ = dp.la_fwd(c["q"], c["k"], c["v"], c["ld"])
    y = dp.group_norm(o, c["w"], c["b"], c["z"])
    gn = dp.group_norm_bwd(o, dy.cuda(), c["w"], c["b"], c["z"])
    gl = dp.la_bwd(c["q"], c["k"], c["v"], gn["x"], c["ld"])
    r = {k: v.double().requires_grad_() for k, v in t.items()}
    S, outs = torch.zeros(B, H, dk, dv, dtype=torch.float64), []
    for i in range(L):
        K, Q = (r[a][:, i].repeat_interleave(H // Hk, 1) for a in ("k", "q"))
        S = S * r["ld"][:, i].exp()[..., None, None] + K[..., :, None] * r["v"][:, i][..., None, :]
        outs.append((S * Q[..., :, None]).sum(-2))
    ro = torch.stack(outs, 1)
    xc = ro - ro.mean(-1, keepdim=True)
    a = xc / (xc.square().mean(-1, keepdim=True) + 1e-5).sqrt() * r["w"] + r["b"]
    ry = a * r["z"] * torch.sigmoid(r["z"])
    ry.backward(dy.double())
    # the norm divides by the readout's spread, which amplifies the fp32 error of small
    # rows: 1e-4 of the norm for both
    got = dict(y=y, q=gl["q"], k=gl["k"], v=gl["v"], ld=gl["ld"], w=gn["weight"], b=gn["bias"], z=gn["gate"])
    for k, g in got.items():
        ref = f64(ry if k == "y" else r[k].grad)
        rel = np.linalg.norm(f64(g) - ref) / np.linalg.norm(ref)
        say(f"  layer {k}: rel {rel:.2e}")
        assert rel <= 1e-4, k


def test_rows_past_32_bit_offsets():
    """More than 2^32 elements: the last rows equal the same rows on their own (a row's
    result does not depend on the others; the weight's gradient does, and is the sum)."""
    G, D, tail = 16, 130, 37
    rows = 2 ** 32 // (G * D) + 100
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(G, D, generator=gen, device="cuda")
    x, dy = (torch.zeros(rows, G, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (x, dy):
        t[-tail:] = torch.randn(tail, G, D, generator=gen, device="cuda")
    last = lambda t: t[-tail:].clone()
    y = dp.group_norm(x, w, silu=True)
    assert torch.equal(last(y), dp.group_norm(last(x), w, silu=True)) and float(y[:-tail].abs().max()) == 0.0
    del y
    g, h = dp.group_norm_bwd(x, dy, w, silu=True), dp.group_norm_bwd(last(x), last(dy), w, silu=True)
    assert torch.equal(last(g["x"]), h["x"]) and float(g["x"][:-tail].abs().max()) == 0.0
    # both sum the same 37 terms and zeros, in another order: 37 roundings of 2^-24 each
    a, b = g["weight"].double(), h["weight"].double()
    assert float((a - b).norm() / b.norm()) <= 2 * 37 * 2.0 ** -24
