"""GPU tests of linear attention with a decay per head (prompt, gradient, single
tokens against a pool) against the recurrence in 64 bits, token by token.

Tolerances, relative to the 2-norm of the tensor, before any run:

* fp32 results (states, their gradients, gradients of the log decays, fp32 inputs):
  every product is fp32 or a three-term bf16 split (2^-24 a term) and every sum has at
  most a few hundred fp32 additions between fp64 or fp32 carries, each off by 2^-24 of
  a partial sum: 64 * 2^-24 = 4e-6 for sums of same-size terms, taken as 1e-5 with
  the cancellation in q . dq - k . dk;
* bf16 results: one rounding, at most half a step of 2^-8 relative per element, and
  the two-term splits (2^-17): 2^-8 = 3.9e-3.
Element by element the difference is at most 2^-8 |x| for the rounding plus 40 times
the 2-norm bound of the fp32 part, relative to the tensor's RMS.
"""
import numpy as np
import pytest
import torch

import linear_rnn_sequence_amd as dp
from parity import f64, say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
F32_TOL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    dp.load()


def recurrence(q, k, v, ld, h0, dout=None, dfinal=None):
    """The definition in fp64 on one sequence: q, k [L,Hk,dk], v [L,H,dv], ld [L,H] or
    None, h0 [H,dk,dv].  Returns out, final and, for dout, the gradients by the
    reverse recurrence (the decay's as <dS_t, e^ld S_{t-1}>, no sums of differences)."""
    L, Hk, dk = q.shape
    H, dv = v.shape[1:]
    r = H // Hk
    Q, K = np.repeat(q, r, axis=1), np.repeat(k, r, axis=1)
    with np.errstate(over="ignore"):
        g = np.ones((L, H)) if ld is None else np.exp(ld)
    S = h0.copy()
    Ss, out = [S], np.zeros((L, H, dv))
    for t in range(L):
        S = g[t][:, None, None] * S + K[t][:, :, None] * v[t][:, None, :]
        Ss.append(S)
        out[t] = np.einsum("hkv,hk->hv", S, Q[t])
    if dout is None:
        return out, S
    dQ, dK, dV, dl = np.zeros_like(Q), np.zeros_like(K), np.zeros_like(v), np.zeros((L, H))
    D = np.zeros_like(S) if dfinal is None else dfinal.copy()
    for t in range(L - 1, -1, -1):
        D = D + Q[t][:, :, None] * dout[t][:, None, :]
        dQ[t] = np.einsum("hkv,hv->hk", Ss[t + 1], dout[t])
        dK[t] = np.einsum("hkv,hv->hk", D, v[t])
        dV[t] = np.einsum("hkv,hk->hv", D, K[t])
        D = g[t][:, None, None] * D
        dl[t] = (D * Ss[t]).sum((1, 2))
    fold = lambda x: x.reshape(L, Hk, r, dk).sum(2)
    return out, S, dict(q=fold(dQ), k=fold(dK), v=dV, ld=dl, h0=D)


def make(B, H, Hk, L, dk, dv, dtype, decay, seed, lens=None, h0=True, scale=1.0):
    """CPU inputs: [B, L, ..], or packed [L, ..] when lens is given."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    lead = (L,) if lens is not None else (B, L)
    x = dict(q=n(*lead, Hk, dk) * dk ** -0.5, k=n(*lead, Hk, dk), v=n(*lead, H, dv) * scale, dout=n(*lead, H, dv))
    x = {a: t.to(DT[dtype]) for a, t in x.items()}
    if decay == "token":
        x["ld"] = -torch.nn.functional.softplus(n(*lead, H) + torch.linspace(-6, 1, H))
    elif decay == "head":
        x["ld"] = torch.log1p(-torch.exp2(-torch.linspace(1.2, 7.0, H)))
    elif decay == "strong":
        x["ld"] = -20.0 * torch.rand(*lead, H, generator=gen)
    else:
        x["ld"] = None
    x["h0"] = n(B, H, dk, dv) * 0.5 if h0 else None
    x["dfinal"] = n(B, H, dk, dv) * 0.5 if h0 else None
    if lens is not None:
        x["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    else:
        x["cu"] = None
    return x


def reference(x, bwd=False):
    """The definition over every sequence of `x`; packed rows behind the last are NaN
    in out and zero in the gradients."""
    H = x["v"].shape[-2]
    cu = None if x["cu"] is None else x["cu"].tolist()
    B = x["q"].shape[0] if cu is None else len(cu) - 1
    outs, states, grads = [], [], []
    for d in range(B):
        at = (lambda t: t[d]) if cu is None else (lambda t: t[cu[d]:cu[d + 1]])
        q, k, v, do = (f64(at(x[n])) for n in ("q", "k", "v", "dout"))
        ld = x["ld"]
        ld = None if ld is None else np.broadcast_to(f64(ld), (q.shape[0], H)) if ld.dim() == 1 else f64(at(ld))
        h0 = np.zeros((H, q.shape[2], v.shape[2])) if x["h0"] is None else f64(x["h0"][d])
        r = recurrence(q, k, v, ld, h0, do if bwd else None, None if x["dfinal"] is None else f64(x["dfinal"][d]))
        outs.append(r[0])
        states.append(r[1])
        if bwd:
            grads.append(r[2])
    join = (lambda a: np.stack(a)) if cu is None else (lambda a: np.concatenate(a))
    res = [join(outs), np.stack(states)]
    if bwd:
        g = {n: join([y[n] for y in grads]) for n in ("q", "k", "v", "ld")}
        g["h0"] = np.stack([y["h0"] for y in grads])
        if x["ld"] is not None and x["ld"].dim() == 1:
            g["ld"] = g["ld"].reshape(-1, H).sum(0)
        res.append(g)
    return res


def check(label, got, ref, low=False):
    got = f64(got)
    assert got.shape == ref.shape, (label, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{label}: non-finite"
    if ref.size == 0:
        return
    norm = np.linalg.norm(ref)
    rms = norm / np.sqrt(ref.size)
    rel = np.linalg.norm(got - ref) / norm if norm else np.linalg.norm(got - ref)
    tol = 2.0 ** -8 if low else F32_TOL
    worst = np.max(np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) if low else 0)) / (rms or 1.0)
    say(f"  {label}: rel {rel:.2e} (tol {tol:.1e}), worst element {worst:.2e} of the RMS")
    assert rel <= tol, f"{label}: {rel:.3e} > {tol:.1e}"
    assert worst <= 40 * F32_TOL, f"{label}: element off by {worst:.3e}"


def dev(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def run_fwd(x, **kw):
    d = dev(x)
    out, fs = dp.la_fwd(d["q"], d["k"], d["v"], d["ld"], cu_seqlens=d["cu"], h0=d["h0"], **kw)
    torch.cuda.synchronize()
    return out, fs


def run_bwd(x, **kw):
    d = dev(x)
    g = dp.la_bwd(d["q"], d["k"], d["v"], d["dout"], d["ld"], cu_seqlens=d["cu"], h0=d["h0"], dfinal=d["dfinal"], **kw)
    torch.cuda.synchronize()
    return g


# B, H, Hk, L, dk, dv, decay, h0: lengths around chunk (32, 64) and segment borders, every
# head width, grouped heads, no decay, strong decays
DENSE = [
    (1, 1, 1, 1, 16, 16, "token", True),
    (2, 3, 3, 31, 16, 32, "token", True),
    (1, 2, 2, 64, 32, 16, "head", False),
    (2, 2, 1, 65, 64, 64, "token", True),
    (1, 4, 2, 127, 128, 64, "none", True),
    (1, 2, 2, 257, 64, 128, "strong", True),
    (1, 6, 2, 300, 128, 128, "token", False),
    (3, 4, 1, 130, 32, 128, "head", True),
    (1, 1, 1, 1000, 128, 16, "token", True),
    (1, 2, 1, 2048, 128, 128, "token", True),
]
ids = [f"B{c[0]}H{c[1]}-{c[2]}L{c[3]}d{c[4]}x{c[5]}{c[6]}" for c in DENSE]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", DENSE, ids=ids)
def test_forward(case, dtype):
    B, H, Hk, L, dk, dv, decay, h0 = case
    x = make(B, H, Hk, L, dk, dv, dtype, decay, 11 + L, h0=h0)
    say(f"case la fwd {case} {dtype}")
    out, fs = run_fwd(x)
    ro, rs = reference(x)
    check("out", out, ro, low=dtype == "bf16")
    check("state", fs, rs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", DENSE, ids=ids)
def test_gradient(case, dtype):
    B, H, Hk, L, dk, dv, decay, h0 = case
    x = make(B, H, Hk, L, dk, dv, dtype, decay, 23 + L, h0=h0)
    say(f"case la bwd {case} {dtype}")
    g = run_bwd(x)
    ref = reference(x, bwd=True)[2]
    for n in ("q", "k", "v"):
        check(n, g[n], ref[n], low=dtype == "bf16")
    check("h0", g["h0"], ref["h0"])
    if x["ld"] is not None:
        check("ld", g["ld"], ref["ld"])


# packed lengths: empty sequences at both ends and in the middle, single tokens, chunk
# borders; `behind` rows after the last sequence
PACKED = [
    (1, 1, [5], 0, 16, 16),
    (4, 2, [0, 1, 64, 0, 63, 65, 1, 0], 7, 64, 64),
    (2, 2, [700, 3, 129], 0, 128, 128),
    (3, 1, [1] * 40 + [0] * 3 + [200], 33, 32, 64),
    (16, 4, [900, 0, 1500], 1, 64, 128),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", PACKED, ids=[f"H{c[0]}n{len(c[2])}d{c[4]}" for c in PACKED])
def test_packed(case, dtype):
    H, Hk, lens, behind, dk, dv = case
    T = sum(lens)
    x = make(len(lens), H, Hk, T + behind, dk, dv, dtype, "token", 5 + T, lens=lens)
    say(f"case la packed {case} {dtype}")
    for n in ("q", "k", "v", "ld", "dout"):  # rows of no sequence are never read
        x[n][T:] = float("nan")
    out0 = torch.full((T + behind, H, dv), 7.0, dtype=DT[dtype], device="cuda")
    out, fs = run_fwd(x, out=out0)
    assert bool((out[T:] == 7.0).all()), "rows behind the last sequence were written"
    ro, rs, rg = reference(x, bwd=True)
    check("out", out[:T], ro, low=dtype == "bf16")
    check("state", fs, rs)
    g = run_bwd(x)
    for n in ("q", "k", "v", "ld"):
        assert bool((g[n][T:] == 0).all()), f"gradient {n} of rows behind the last sequence"
        check(n, g[n][:T], rg[n], low=dtype == "bf16" and n != "ld")
    check("h0", g["h0"], rg["h0"])


@pytest.mark.parametrize("cu", [[1, 3, 8], [0, 5, 3], [0, 4, 9], [0, -1, 8]])
def test_broken_offsets_make_every_sequence_empty(cu):
    x = make(2, 2, 2, 8, 16, 16, "f32", "token", 3, lens=[4, 4])
    x["cu"] = torch.tensor(cu, dtype=torch.int32)
    out0 = torch.full((8, 2, 16), 7.0, device="cuda")
    out, fs = run_fwd(x, out=out0)
    assert bool((out == 7.0).all()) and torch.equal(fs.cpu(), x["h0"])
    g = run_bwd(x)
    for n in ("q", "k", "v", "ld"):
        assert bool((g[n] == 0).all())
    assert torch.equal(g["h0"].cpu(), x["dfinal"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_resets_and_infinite_decays(dtype):
    """ld = -inf erases the state exactly: what follows equals a sequence of its own,
    also inside a chunk and after strong decays; its gradient is zero."""
    x = make(1, 2, 2, 200, 64, 64, dtype, "token", 9)
    x["ld"][0, 70] = float("-inf")
    x["ld"][0, 90:100] = -50.0
    x["ld"][0, 128] = float("-inf")
    out, fs = run_fwd(x)
    ro, rs, rg = reference(x, bwd=True)
    check("out", out, ro, low=dtype == "bf16")
    check("state", fs, rs)
    g = run_bwd(x)
    for n in ("q", "k", "v", "h0", "ld"):
        check(n, g[n], rg[n], low=dtype == "bf16" and n in "qkv")
    # the gradient of an erasing decay is exactly zero in the definition; here up to the
    # rounding of the two sums it is the difference of
    assert float(g["ld"][0, [70, 128]].abs().max()) <= 40 * F32_TOL * float(g["ld"].abs().max())


# B, H, L, decay, lens, tokens whose decay erases the state: the first and the last, chunk
# borders of either path, neighbours, in one segment and in many, packed, a whole head
ERASED = [(2, 2, 200, "token", None, [0, 31, 32, 63, 64, 65, 128, 199]), (1, 1, 2500, "token", None, [5, 640, 641, 2499]),
          (3, 2, 400, "token", [250, 0, 150], [0, 100, 249, 250, 399]), (2, 3, 300, "head", None, None)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", ERASED, ids=["one", "many", "packed", "head"])
def test_gradient_of_an_erasing_decay_is_zero(case, dtype):
    """e^ld is 0 from -1000 down, and so is its derivative, exactly; the others' stays the
    definition's."""
    B, H, L, decay, lens, at = case
    x = make(B, H, H, L, 64, 64, dtype, decay, 67, lens=lens)
    if at is None:
        x["ld"][1] = float("-inf")
    else:
        x["ld"][..., at, :] = float("-inf")
        x["ld"][..., at[1], :] = -1000.0
        x["ld"][..., at[2], 0] = -3e38
    g = run_bwd(x)
    zero = x["ld"] <= -1000.0
    assert bool(zero.any()) and bool((g["ld"].cpu()[zero] == 0).all())
    rg = reference(x, bwd=True)[2]
    for n in ("q", "k", "v", "h0", "ld"):
        check(n, g[n], rg[n], low=dtype == "bf16" and n in "qkv")


# sequences without an initial state: B, H, Hk, L, dk, dv, decay, lens; single tokens, a few,
# one and many segments
FIRST = [(5, 2, 1, 1, 128, 32, "token", None), (3, 4, 2, 1, 64, 64, "head", None), (2, 2, 2, 3, 32, 128, "token", None),
         (2, 2, 2, 700, 64, 64, "token", None), (6, 2, 2, 300, 16, 64, "token", [1, 0, 1, 270, 2, 26])]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", FIRST, ids=[f"B{c[0]}L{c[3]}d{c[4]}{c[6]}{'p' if c[7] else ''}" for c in FIRST])
def test_gradient_of_the_first_decay(case, dtype):
    """Nothing precedes a sequence's first token, so its decay's gradient is exactly zero, with
    one decay per head also the sum over sequences of a token; with an initial state it is
    e^ld <h0, D>, to an fp32 product's error of itself where it is the only token."""
    B, H, Hk, L, dk, dv, decay, lens = case
    x = make(B, H, Hk, L, dk, dv, dtype, decay, 71 + L, lens=lens, h0=False)
    g = run_bwd(x)
    rg = reference(x, bwd=True)[2]
    if decay == "head":
        assert bool((g["ld"] == 0).all())
    else:
        at = g["ld"][:, 0] if lens is None else g["ld"][[int(c) for c, n in zip(x["cu"], lens) if n]]
        assert bool((at == 0).all())
    for n in ("q", "k", "v", "ld"):
        check(n, g[n], rg[n], low=dtype == "bf16" and n in "qkv")
    if L == 1:
        y = make(B, H, Hk, L, dk, dv, dtype, decay, 73, h0=True)
        y["h0"] *= 1e-3
        check("ld", run_bwd(y)["ld"], reference(y, bwd=True)[2]["ld"])


# B, H, Hk, L, dk, dv, decay, lens: two to ten tokens, decays down to e^-20, no initial state
SHORT = [(1, 1, 1, 2, 64, 64, "strong", None), (4, 1, 1, 6, 32, 128, "strong", [0, 2, 0, 4]), (6, 4, 2, 2, 64, 64, "strong", None),
         (3, 4, 4, 5, 128, 16, "strong", None), (5, 4, 1, 30, 16, 32, "strong", [2, 10, 3, 15, 0]), (3, 8, 8, 3, 128, 128, "head", None)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SHORT, ids=[f"B{c[0]}L{c[3]}d{c[4]}{c[6]}{'p' if c[7] else ''}" for c in SHORT])
def test_decay_gradient_of_short_sequences(case, dtype):
    """Only pairs of different tokens enter it, far smaller than a token's own term when they
    are few or the decays strong: an fp32 result's error relative to itself all the same."""
    B, H, Hk, L, dk, dv, decay, lens = case
    for seed in range(5):
        x = make(B, H, Hk, L, dk, dv, dtype, decay, 79 + seed, lens=lens, h0=False)
        check("ld", run_bwd(x)["ld"], reference(x, bwd=True)[2]["ld"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_against_differences(dtype):
    """Directional derivatives of the fp64 definition by central differences."""
    x = make(1, 2, 1, 90, 32, 32, dtype, "token", 77)
    g = run_bwd(x)
    gen = torch.Generator().manual_seed(1)
    w, wf = f64(x["dout"]), f64(x["dfinal"])

    def loss(y):
        o, s = reference(y)
        return float((o * w).sum() + (s * wf).sum())

    for n in ("q", "k", "v", "ld", "h0"):
        u = torch.randn(x[n].shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        hi, lo = dict(x), dict(x)
        hi[n], lo[n] = x[n].double() + e * u, x[n].double() - e * u
        fd = (loss(hi) - loss(lo)) / (2 * e)
        an = float((f64(g[n]) * u.numpy()).sum())
        size = float(np.linalg.norm(f64(g[n])))
        # the rounding of g projects on a random direction: 2^-8 (bf16) or 1e-5 of |g|; the
        # differences' own error is far below
        tol = (2.0 ** -8 if dtype == "bf16" and n in "qkv" else 1e-5) * 4 * size + 1e-6 * size
        say(f"  d{n}: {an:.6f} against {fd:.6f} (|g| {size:.2f})")
        assert abs(an - fd) <= tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_and_split_resume(dtype):
    """The same call gives the same bits; a sequence cut in two, its state passed on in
    place, gives the whole one's results to fp32 rounding."""
    x = make(2, 4, 2, 500, 64, 64, dtype, "token", 31)
    out, fs = run_fwd(x)
    out2, fs2 = run_fwd(x)
    assert torch.equal(out, out2) and torch.equal(fs, fs2)
    g, g2 = run_bwd(x), run_bwd(x)
    assert all(torch.equal(g[n], g2[n]) for n in g)
    d = dev(x)
    st = d["h0"].clone()
    parts = []
    for a, b in ((0, 173), (173, 500)):
        c = lambda n: d[n][:, a:b].contiguous()
        o, s = dp.la_fwd(c("q"), c("k"), c("v"), c("ld"), h0=st, final_state=st)
        assert s is st
        parts.append(o)
    ro, rs = reference(x)
    check("out", torch.cat(parts, 1), ro, low=dtype == "bf16")
    check("state", st, rs)


def test_fp32_out_of_bf16_inputs():
    x = make(1, 2, 2, 333, 128, 128, "bf16", "token", 41)
    out, fs = run_fwd(x, out_dtype=torch.float32)
    ro, rs = reference(x)
    assert out.dtype == torch.float32
    check("out", out, ro)
    check("state", fs, rs)


# B, H, Hk, L, dk, dv, lens: one segment, several, packed and grouped
ASKED = [(2, 2, 1, 200, 64, 64, None), (1, 2, 2, 1500, 128, 128, None), (1, 3, 3, 700, 32, 128, None),
         (3, 4, 2, 1300, 128, 64, [900, 0, 400])]


@pytest.mark.parametrize("case", ASKED, ids=[f"B{c[0]}H{c[1]}L{c[3]}d{c[4]}x{c[5]}" for c in ASKED])
def test_results_do_not_depend_on_what_else_is_asked_for(case):
    """A bf16 result is the fp32 one rounded once: out is DP_OUT_F32's out rounded, with
    and without the final state, and dq, dk, dv have the same bits with and without the
    gradients of the decays and of the initial state."""
    B, H, Hk, L, dk, dv, lens = case
    x = make(B, H, Hk, L, dk, dv, "bf16", "token", 59, lens=lens)
    out, fs = run_fwd(x)
    full, fs32 = run_fwd(x, out_dtype=torch.float32)
    alone, none = run_fwd(x, return_state=False)
    assert none is None and torch.equal(out, full.bfloat16()) and torch.equal(out, alone) and torch.equal(fs, fs32)
    g = run_bwd(x)
    for left in (["ld"], ["h0"], ["ld", "h0"]):
        part = run_bwd(x, grads={n: None for n in left})
        assert all(part[n] is None if n in left else torch.equal(g[n], part[n]) for n in g), left
    with pytest.raises(dp.DPError):
        run_bwd(x, grads=dict(q=None))


@pytest.mark.parametrize("case", ASKED, ids=[f"B{c[0]}H{c[1]}L{c[3]}d{c[4]}x{c[5]}" for c in ASKED])
def test_bf16_results_are_rounded_fp32_results(case):
    """Element by element at most half a bf16 step off the definition, and an fp32
    result's error: 64 * 2^-24 of the tensor's RMS (64 sums of 2^-24 of a partial sum each,
    see the top; two-term operands would leave 2^-18 of every product)."""
    B, H, Hk, L, dk, dv, lens = case
    x = make(B, H, Hk, L, dk, dv, "bf16", "token", 61, lens=lens)
    out, _ = run_fwd(x)
    g = run_bwd(x)
    ro, _, rg = reference(x, bwd=True)
    for n, got, ref in [("out", out, ro)] + [(n, g[n], rg[n]) for n in "qkv"]:
        half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(ref), 1e-30))) - 8)
        over = np.max(np.abs(f64(got) - ref) - half) / np.sqrt(np.mean(ref * ref))
        say(f"  {n}: {over:.2e} of the RMS past half a step")
        assert over <= 64 * 2.0 ** -24, n


def test_large_and_small_values():
    """The bf16 path has bf16's range: values far outside fp16's."""
    for scale in (1e8, 1e-8):
        x = make(1, 1, 1, 150, 64, 64, "bf16", "token", 43, scale=scale, h0=False)
        out, fs = run_fwd(x)
        ro, rs = reference(x)
        check("out", out, ro, low=True)
        check("state", fs, rs)


def test_non_finite_values_stay_in_their_head_and_sequence():
    x = make(2, 2, 2, 200, 32, 32, "bf16", "token", 47)
    x["v"][0, 100, 1, 3] = float("inf")
    out, fs = run_fwd(x)
    ro, rs = reference(x)
    o = f64(out)
    assert not np.isfinite(o[0, 100:, 1, 3]).any() and not np.isfinite(f64(fs)[0, 1, :, 3]).any()
    good = np.ones_like(o, bool)
    good[0, 64:, 1, 3] = False  # the chunk that holds token 100, and what follows
    assert np.isfinite(o[good]).all()
    assert np.max(np.abs(o[good] - ro[good]) / (np.abs(ro[good]) + 1)) < 2.0 ** -7


def test_empty_batch_passes_the_state_on():
    x = make(2, 2, 1, 0, 16, 32, "f32", "token", 3)
    out, fs = run_fwd(x)
    assert out.shape == (2, 0, 2, 32) and torch.equal(fs.cpu(), x["h0"])
    g = run_bwd(x)
    assert torch.equal(g["h0"].cpu(), x["dfinal"])


# ------------------------------------------------------------------ single tokens


def decode_ref(x, state, slots):
    """Rows in batch order on copies of the states, fp64."""
    st, out = f64(state).copy(), np.zeros(x["v"].shape)
    H, Hk = x["v"].shape[1], x["q"].shape[1]
    for b in range(x["q"].shape[0]):
        s = b if slots is None else slots[b]
        if not 0 <= s < st.shape[0]:
            continue
        q, k = (np.repeat(f64(x[n][b]), H // Hk, axis=0) for n in ("q", "k"))
        if x["ld"] is not None:
            st[s] *= np.exp(f64(x["ld"] if x["ld"].dim() == 1 else x["ld"][b]))[:, None, None]
        st[s] += k[:, :, None] * f64(x["v"][b])[:, None, :]
        out[b] = np.einsum("hkv,hk->hv", st[s], q)
    return out, st


# B, H, Hk, dk, dv, slots (None: identity; entries outside the pool are padding), decay
DECODE = [
    (1, 1, 1, 16, 16, None, "token"),
    (3, 4, 2, 64, 32, [2, 0, 4], "token"),
    (5, 3, 1, 128, 128, [4, -1, 0, 99, 2], "head"),
    (6, 2, 2, 32, 64, [1, 3, 1, 1, -1, 3], "token"),   # one slot in several rows
    (4, 8, 8, 16, 128, [3, 2, 1, 0], "none"),
    (300, 2, 1, 64, 64, "random", "token"),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", DECODE, ids=[f"B{c[0]}H{c[1]}-{c[2]}d{c[3]}x{c[4]}" for c in DECODE])
def test_decode(case, dtype):
    B, H, Hk, dk, dv, slots, decay = case
    say(f"case la decode {case} {dtype}")
    x = make(1, H, Hk, B, dk, dv, dtype, decay, B + dk, lens=[B])
    n = 40 if slots == "random" else max(5, B)
    if slots == "random":  # many rows of one slot, some of none
        slots = np.random.RandomState(0).randint(-3, n + 3, B).tolist()
    state = torch.randn(n, H, dk, dv, generator=torch.Generator().manual_seed(2))
    st = state.clone().cuda()
    out = torch.full((B, H, dv), 7.0, dtype=DT[dtype], device="cuda")
    d = dev(x)
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    dp.la_decode(d["q"], d["k"], d["v"], st, d["ld"], slots=sl, out=out)
    torch.cuda.synchronize()
    ro, rs = decode_ref(x, state, slots)
    live = [b for b in range(B) if slots is None or 0 <= slots[b] < n]
    dead = [b for b in range(B) if b not in live]
    check("out", out[live], ro[live], low=dtype == "bf16")
    check("state", st, rs)
    assert bool((out[dead] == 7.0).all()), "a padding row was written"
    untouched = [s for s in range(n) if slots is not None and s not in slots]
    assert torch.equal(st[untouched].cpu(), state[untouched])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_then_decode(dtype):
    """A packed prefill into the pool's slots, then one launch per token: every output
    and the final states equal the definition over the whole sequences."""
    lens, K = [70, 1, 129], 9
    B, H, Hk, dk, dv = 3, 4, 2, 64, 64
    full = make(B, H, Hk, max(lens) + K, dk, dv, dtype, "token", 13)
    pool = torch.zeros(1, 5, H, dk, dv, device="cuda")
    slots = [4, 0, 2]
    d = dev(full)
    pk = lambda n: torch.cat([d[n][i, :lens[i]] for i in range(B)]).contiguous()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    _, fs = dp.la_fwd(pk("q"), pk("k"), pk("v"), pk("ld"), cu_seqlens=cu, h0=d["h0"])
    pool[0, slots] = fs
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
    outs = []
    for t in range(K):
        row = lambda n: torch.stack([d[n][i, lens[i] + t] for i in range(B)]).contiguous()
        outs.append(dp.la_decode(row("q"), row("k"), row("v"), pool[0], row("ld"), slots=sl))
    torch.cuda.synchronize()
    got = torch.stack(outs, 1)
    for i in range(B):
        L = lens[i] + K
        ro, rs = recurrence(*(f64(full[n][i, :L]) for n in ("q", "k", "v", "ld")), f64(full["h0"][i]))
        check(f"out {i}", got[i], ro[lens[i]:], low=dtype == "bf16")
        check(f"state {i}", pool[0, slots[i]], rs)


# ------------------------------------------------------------------ how it is called


def test_other_stream_and_captured_replays():
    """Forward, gradient and decode on a side stream, and captured into graphs that are
    replayed on new inputs in the same buffers, eager work between the replays."""
    xs = [make(2, 4, 2, 200, 64, 64, "bf16", "token", s) for s in (1, 2, 3)]
    d = dev(xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, fs = dp.la_fwd(d["q"], d["k"], d["v"], d["ld"], h0=d["h0"], stream=side)
    side.synchronize()
    want, wfs = dp.la_fwd(d["q"], d["k"], d["v"], d["ld"], h0=d["h0"])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(fs, wfs)
    state = torch.zeros(2, 4, 64, 64, device="cuda")
    first = lambda n: d[n][:, 0].contiguous()
    tok = {n: first(n) for n in ("q", "k", "v", "ld")}

    def step():
        o, s = dp.la_fwd(d["q"], d["k"], d["v"], d["ld"], h0=d["h0"])
        g = dp.la_bwd(d["q"], d["k"], d["v"], d["dout"], d["ld"], h0=d["h0"], dfinal=d["dfinal"])
        state.copy_(s)
        return o, s, g, dp.la_decode(tok["q"], tok["k"], tok["v"], state, tok["ld"])

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        co, cs, cg, cd = step()
    for x in (*xs, xs[1]):
        for n in ("q", "k", "v", "ld", "dout", "h0", "dfinal"):
            d[n].copy_(x[n])
        for n in tok:
            tok[n].copy_(d[n][:, 0])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (co, cs, cd, *(cg[n] for n in sorted(cg)))]
        o, s, g, dd = step()
        torch.cuda.synchronize()
        for a, b in zip(got, [o, s, dd, *(g[n] for n in sorted(g))]):
            assert torch.equal(a, b)


def test_given_workspace_and_outputs():
    x = make(1, 2, 2, 700, 64, 64, "f32", "token", 8)
    d = dev(x)
    n = dp.la_fwd_workspace_size(1, 2, 2, 700, 64, 64)
    assert n > 0
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(d["v"])
    o, fs = dp.la_fwd(d["q"], d["k"], d["v"], d["ld"], h0=d["h0"], out=out, workspace=ws[:n])
    torch.cuda.synchronize()
    assert o is out and bool((ws[n:] == 255).all())
    check("out", out, reference(x)[0])
    nb = dp.la_bwd_workspace_size(1, 2, 2, 700, 64, 64)
    wb = torch.full((nb + 64,), 255, dtype=torch.uint8, device="cuda")
    g = dp.la_bwd(d["q"], d["k"], d["v"], d["dout"], d["ld"], h0=d["h0"], dfinal=d["dfinal"], workspace=wb[:nb])
    torch.cuda.synchronize()
    assert bool((wb[nb:] == 255).all())
    check("q", g["q"], reference(x, bwd=True)[2]["q"])
    with pytest.raises(dp.DPError) as e:
        dp.la_fwd(d["q"], d["k"], d["v"], d["ld"], workspace=ws[:n - 256])
    assert e.value.code == dp.binding.DP_EWORKSPACE


# L that is cut into one segment, a few (added up in the walk) and many (scanned first),
# one length and packed
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 2, 100, None, 64), (2, 2, 700, None, 64), (1, 1, 3000, None, 32),
                                  (4, 8, 2500, [900, 0, 40, 1500, 60], 128)], ids=["one", "few", "many", "packed"])
def test_state_passed_on_in_place(case, dtype):
    """h0 and final_state in one buffer give what two buffers give, bit for bit."""
    B, H, L, lens, d = case
    if lens is not None:
        B = len(lens)
    x = make(B, H, H, L, d, d, dtype, "head", 6, lens=lens)
    out, fs = run_fwd(x)
    y = dev(x)
    st = y["h0"].clone()
    o, s = dp.la_fwd(y["q"], y["k"], y["v"], y["ld"], cu_seqlens=y["cu"], h0=st, final_state=st)
    torch.cuda.synchronize()
    assert s is st and torch.equal(o, out) and torch.equal(st, fs)
    if lens is None:
        check("state", st, reference(x)[1])


# ------------------------------------------------------------------ more of how it is cut

# B, H, Hk, L, dk, dv, decay, lens: gradients over one to three segments (added up in the
# walks) and over many (scanned first), forwards over more than sixteen; odd numbers of
# (segment, key head) groups; one decay per head over packed and grouped heads
CUTS = [
    (1, 1, 1, 300, 64, 64, "token", None),
    (1, 3, 1, 1201, 32, 16, "head", None),
    (1, 5, 1, 2500, 64, 64, "none", None),
    (1, 6, 3, 1500, 128, 128, "head", None),
    (7, 10, 5, 129, 64, 128, "token", None),
    (3, 9, 3, 1200, 128, 32, "head", [1, 1100, 99]),
    (5, 2, 2, 1700, 32, 64, "none", [0, 800, 0, 900, 0]),
    (1, 4, 1, 2300, 16, 128, "strong", [2300]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CUTS, ids=[f"B{c[0]}H{c[1]}-{c[2]}L{c[3]}d{c[4]}x{c[5]}{c[6]}" for c in CUTS])
def test_cuts(case, dtype):
    B, H, Hk, L, dk, dv, decay, lens = case
    x = make(B, H, Hk, L, dk, dv, dtype, decay, 7 * L + H, lens=lens)
    say(f"case la cut {case} {dtype}")
    out, fs = run_fwd(x)
    g = run_bwd(x)
    ro, rs, rg = reference(x, bwd=True)
    check("out", out, ro, low=dtype == "bf16")
    check("state", fs, rs)
    for n in ("q", "k", "v", "h0") + (() if x["ld"] is None else ("ld",)):
        check(n, g[n], rg[n], low=dtype == "bf16" and n in "qkv")


# B, H, Hk, L, dk, dv, decay, lens with many segments, on both sides of the rule for who adds
# their states up: forwards and gradients of wide heads (the scan) and of narrow ones (the
# walks, the decays' gradient too), of one length and packed with cut, uncut and empty
# sequences side by side
SIDES = [
    (1, 4, 4, 2500, 128, 128, "token", None),
    (2, 2, 1, 1300, 128, 64, "head", None),
    (1, 2, 2, 2500, 32, 32, "token", None),
    (1, 3, 1, 2000, 16, 64, "head", None),
    (5, 2, 2, 2700, 128, 128, "token", [1700, 0, 40, 900, 60]),
    (5, 3, 1, 2700, 128, 128, "head", [60, 900, 40, 0, 1700]),
    (5, 2, 2, 2700, 64, 64, "head", [1700, 0, 40, 900, 60]),
    (3, 2, 1, 1500, 32, 16, "token", [1400, 1, 99]),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_around_the_first_cut(d, dtype):
    """Walked alone, and cut into segments of a chunk."""
    for L in (128, 129, 192, 193, 256, 257):
        x = make(1, 2, 1, L, d, d, dtype, "token", L)
        out, fs = run_fwd(x)
        g = run_bwd(x)
        ro, rs, rg = reference(x, bwd=True)
        check(f"out {L}", out, ro, low=dtype == "bf16")
        check(f"state {L}", fs, rs)
        for n in ("q", "k", "v", "h0", "ld"):
            check(f"{n} {L}", g[n], rg[n], low=dtype == "bf16" and n in "qkv")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SIDES, ids=[f"H{c[1]}-{c[2]}L{c[3]}d{c[4]}x{c[5]}{c[6]}{'p' if c[7] else ''}" for c in SIDES])
def test_many_segments(case, dtype):
    """Results against the definition, and the state passed on in one buffer, bit for bit
    what two buffers give."""
    B, H, Hk, L, dk, dv, decay, lens = case
    x = make(B, H, Hk, L, dk, dv, dtype, decay, 3 * L + H, lens=lens)
    say(f"case la many {case} {dtype}")
    out, fs = run_fwd(x)
    y = dev(x)
    st = y["h0"].clone()
    o, _ = dp.la_fwd(y["q"], y["k"], y["v"], y["ld"], cu_seqlens=y["cu"], h0=st, final_state=st)
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(st, fs)
    g = run_bwd(x)
    ro, rs, rg = reference(x, bwd=True)
    check("out", out, ro, low=dtype == "bf16")
    check("state", fs, rs)
    for n in ("q", "k", "v", "h0", "ld"):
        check(n, g[n], rg[n], low=dtype == "bf16" and n in "qkv")


def test_calls_side_by_side():
    """Two streams with calls in flight at once, and two graphs of different inputs replayed
    on them together: each gives what it gives alone."""
    xs = [dev(make(2, 4, 2, 900, 64, 64, "bf16", "token", s)) for s in (1, 2)]

    def step(d):
        o, s = dp.la_fwd(d["q"], d["k"], d["v"], d["ld"], h0=d["h0"])
        g = dp.la_bwd(d["q"], d["k"], d["v"], d["dout"], d["ld"], h0=d["h0"], dfinal=d["dfinal"])
        return [o, s, *(g[n] for n in sorted(g))]

    want = [step(d) for d in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(xs[i]))
    torch.cuda.synchronize()
    graphs = []
    for d in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r = step(d)
        graphs.append((graph, r))
    for _ in range(3):
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for i, (_, r) in enumerate(graphs):
            got[i].append([t.clone() for t in r])
        torch.cuda.synchronize()
    for i in (0, 1):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_rows_past_32_bit_offsets():
    """Value rows of more than 2^32 elements: the last sequence of a packed batch equals
    the definition over its own rows, forwards and backwards."""
    H, dk, dv, tail = 128, 16, 128, 70
    T = 2 ** 32 // (H * dv) + 500
    x = make(1, H, 1, tail, dk, dv, "bf16", "token", 3, lens=[tail])
    big = {n: torch.zeros((T, *x[n].shape[1:]), dtype=x[n].dtype, device="cuda") for n in ("q", "k", "v", "ld", "dout")}
    for n in big:
        big[n][-tail:] = x[n].cuda()
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    h0, df = (torch.cat([torch.zeros_like(x[n]), x[n]]).cuda() for n in ("h0", "dfinal"))
    out, fs = dp.la_fwd(big["q"], big["k"], big["v"], big["ld"], cu_seqlens=cu, h0=h0)
    ro, rs, rg = reference(x, bwd=True)
    check("out", out[-tail:], ro, low=True)
    check("state", fs[1:], rs)
    assert float(out[:-tail].abs().max()) == 0.0 and float(fs[0].abs().max()) == 0.0
    del out
    g = dp.la_bwd(big["q"], big["k"], big["v"], big["dout"], big["ld"], cu_seqlens=cu, h0=h0, dfinal=df)
    for n in ("q", "k", "v", "ld"):
        check(n, g[n][-tail:], rg[n], low=n != "ld")
    check("h0", g["h0"][1:], rg["h0"])
    assert float(g["v"][:-tail].abs().max()) == 0.0


def test_decode_slots_past_32_bit_offsets():
    H, d = 4, 128
    n = 2 ** 32 // (H * d * d) + 3  # a pool of more than 2^32 floats
    x = make(1, H, H, 2, d, d, "bf16", "token", 5, lens=[2])
    pool = torch.zeros(n, H, d, d, device="cuda")
    state = torch.randn(2, H, d, d, generator=torch.Generator().manual_seed(2))
    pool[0], pool[n - 1] = state[0].cuda(), state[1].cuda()
    y = dev(x)
    out = dp.la_decode(y["q"], y["k"], y["v"], pool, y["ld"], slots=torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda"))
    ro, rs = decode_ref(x, state, [1, 0])
    check("out", out, ro, low=True)
    check("state", pool[[0, n - 1]], rs)
    assert float(pool[1:n - 1].amax()) == 0.0 and float(pool[1:n - 1].amin()) == 0.0
