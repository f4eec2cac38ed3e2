"""CPU tests of linear attention's, the group norm's and the state pages' refusals:
every check answers on the host before any HIP call, so none needs a GPU."""
import ctypes

import pytest
import torch

import linear_rnn_sequence_amd as dp
from linear_rnn_sequence_amd import binding

E = binding
P = 1 << 20  # an aligned non-null address; the checks fail before any use
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(binding.LIB_PATH):
        from linear_rnn_sequence_amd import build as b
        b.build()
    return dp.load()


def la_fwd(lib, suf, q=P, k=P, v=P, ld=P, cu=None, B=2, H=4, Hk=2, L=10, dk=64, dv=64, out=P, fs=P, h0=P, ws=P, wsb=BIG,
           flags=0):
    return getattr(lib, f"dp_la_fwd_{suf}")(q, k, v, ld, cu, B, H, Hk, L, dk, dv, out, fs, h0, ws, wsb, flags, None)


def la_bwd(lib, suf, q=P, k=P, v=P, ld=P, cu=None, h0=P, dout=P, dfinal=P, B=2, H=4, Hk=2, L=10, dk=64, dv=64, dq=P, dk_=P,
           dv_=P, dld=P, dh0=P, ws=P, wsb=BIG, flags=0):
    return getattr(lib, f"dp_la_bwd_{suf}")(q, k, v, ld, cu, h0, dout, dfinal, B, H, Hk, L, dk, dv, dq, dk_, dv_, dld, dh0,
                                            ws, wsb, flags, None)


def la_decode(lib, suf, q=P, k=P, v=P, ld=P, slots=P, B=2, H=4, Hk=2, n=3, dk=64, dv=64, out=P, state=P, flags=0):
    return getattr(lib, f"dp_la_decode_{suf}")(q, k, v, ld, slots, B, H, Hk, n, dk, dv, out, state, flags, None)


SIZES = [(dict(B=0), E.DP_EINVAL), (dict(H=0), E.DP_EINVAL), (dict(Hk=0), E.DP_EINVAL), (dict(Hk=3), E.DP_EINVAL),
         (dict(Hk=8), E.DP_EINVAL), (dict(dk=24), E.DP_ENOTSUP), (dict(dv=256), E.DP_ENOTSUP), (dict(dk=0), E.DP_EINVAL)]


@pytest.mark.parametrize("suf", ["f32", "bf16"])
def test_linear_attention_checks(lib, suf):
    for kw, code in SIZES:
        assert la_fwd(lib, suf, **kw) == code, kw
        assert la_bwd(lib, suf, **kw) == code, kw
        assert la_decode(lib, suf, **kw) == code, kw
    for fn in (la_fwd, la_bwd):
        assert fn(lib, suf, L=-1) == E.DP_EINVAL
        assert fn(lib, suf, L=2 ** 30, B=4) == E.DP_ENOTSUP      # rows past 32 bits
        assert fn(lib, suf, flags=E.LA_HEAD_DECAY, ld=None, **(dict(dld=None) if fn is la_bwd else {})) == E.DP_EINVAL
        assert fn(lib, suf, flags=64) == E.DP_EINVAL
        assert fn(lib, suf, L=100000, ws=None) == E.DP_EWORKSPACE
        assert fn(lib, suf, L=100000, wsb=100) == E.DP_EWORKSPACE
        assert fn(lib, suf, L=100000, ws=P + 16) == E.DP_EWORKSPACE
        assert fn(lib, suf, cu=P, ws=None) == E.DP_EWORKSPACE   # the segment table
        assert fn(lib, suf, cu=P + 2) == E.DP_EINVAL
        for n in ("q", "k", "v"):
            assert fn(lib, suf, **{n: None}) == E.DP_EINVAL
            assert fn(lib, suf, **{n: P + 8}) == E.DP_EINVAL
        assert fn(lib, suf, h0=P + 4) == E.DP_EINVAL
    for n in ("out",):
        assert la_fwd(lib, suf, **{n: None}) == E.DP_EINVAL
    assert la_fwd(lib, suf, fs=P + 8) == E.DP_EINVAL
    for n in ("dout", "dq", "dk_", "dv_"):
        assert la_bwd(lib, suf, **{n: None}) == E.DP_EINVAL
        assert la_bwd(lib, suf, **{n: P + 8}) == E.DP_EINVAL
    assert la_bwd(lib, suf, ld=None) == E.DP_EINVAL             # dld without ld
    assert la_bwd(lib, suf, flags=E.OUT_F32) == E.DP_EINVAL
    for n in ("q", "k", "v", "out", "state"):
        assert la_decode(lib, suf, **{n: None}) == E.DP_EINVAL
    assert la_decode(lib, suf, slots=None, B=4) == E.DP_EINVAL   # more rows than states
    assert la_decode(lib, suf, n=0) == E.DP_EINVAL
    assert la_decode(lib, suf, flags=1) == E.DP_EINVAL
    assert la_decode(lib, suf, state=P + 4) == E.DP_EINVAL


def test_linear_attention_workspace_sizes(lib):
    # one segment per sequence needs nothing when the lengths are known ...
    assert dp.la_fwd_workspace_size(1, 8, 8, 37, 64, 64) == 0
    # ... and the segment table and order when they are packed: 8 + 2 and 8 ints
    assert dp.la_fwd_workspace_size(8, 8, 8, 37, 64, 64, packed=True) == 512
    # cut sequences: an fp32 state and a decay per segment and head
    n = dp.la_fwd_workspace_size(4, 16, 16, 4096, 128, 128)
    segs, rest = divmod(n, 16 * (128 * 128 * 4 + 4))
    assert n > 0 and segs % 4 == 0 and rest == 0
    with pytest.raises(dp.DPError):
        dp.la_fwd_workspace_size(1, 3, 2, 10, 64, 64)
    out = ctypes.c_size_t(0)
    assert lib.dp_la_bwd_workspace_size(1, 1, 1, 1, 16, 16, 0, None) == E.DP_EINVAL
    assert lib.dp_la_bwd_workspace_size(1, 1, 1, 1, 16, 17, 0, ctypes.byref(out)) == E.DP_ENOTSUP


def test_short_sequences_are_not_cut(lib):
    """Alone up to two chunks of a wide state, three of a narrow one; cut ones need states."""
    for d, alone in ((128, 128), (64, 192), (16, 192)):
        assert dp.la_fwd_workspace_size(1, 8, 8, alone, d, d) == 0
        assert dp.la_fwd_workspace_size(1, 8, 8, alone + 1, d, d) >= 2 * 8 * d * d * 4


def test_longest_sequences_are_cut_as_short_ones(lib):
    """Two thousand million tokens of a head: a state and a decay per segment, about as
    many segments as for a tenth of them (a length near 2^31 plus a segment passes 32 bits)."""
    for H, sizes in ((1, (200_000_000, 2_000_000_000, 2 ** 31 - 1000)), (300, (200_000_000, 2_000_000_000))):
        for fn in (dp.la_fwd_workspace_size, ):
            got = [fn(1, H, H, L, 16, 16) for L in sizes]
            assert got[0] > 0 and all(abs(g - got[0]) <= got[0] // 50 for g in got), (H, got)
    with pytest.raises(dp.DPError):
        dp.la_fwd_workspace_size(1, 1, 1, 2 ** 31 - 1, 16, 16)


@pytest.mark.parametrize("suf", ["f32", "bf16"])
def test_overlaps_are_refused(lib, suf):
    """Every buffer at an address of its own but for one pair, one element inside the other;
    the pair that may be one buffer is no exception when it is shifted."""
    at = lambda i: (i + 1) << 32
    fwd = dict(zip(("q", "k", "v", "ld", "out", "fs", "h0", "ws"), map(at, range(8))))
    for a in ("out", "fs", "ws"):
        for b in fwd:
            if a != b and (a, b) != ("fs", "h0"):
                assert la_fwd(lib, suf, L=1000, **{**fwd, a: fwd[b] + 256, "wsb": BIG}) == E.DP_EINVAL, (a, b)
    assert la_fwd(lib, suf, L=1000, **{**fwd, "fs": fwd["h0"] + 256}) == E.DP_EINVAL
    bwd = dict(zip(("q", "k", "v", "ld", "h0", "dout", "dfinal", "dq", "dk_", "dv_", "dld", "dh0", "ws"), map(at, range(13))))
    for a in ("dq", "dk_", "dv_", "dh0", "ws"):
        for b in bwd:
            if a != b and b not in ("ld", "dld"):
                assert la_bwd(lib, suf, L=1000, **{**bwd, a: bwd[b] + 256}) == E.DP_EINVAL, (a, b)
    assert la_bwd(lib, suf, L=1000, **{**bwd, "dld": bwd["ld"] + 4}) == E.DP_EINVAL
    assert la_bwd(lib, suf, L=1000, **{**bwd, "dh0": bwd["dfinal"]}) == E.DP_EINVAL
    dec = dict(zip(("q", "k", "v", "ld", "slots", "out", "state"), map(at, range(7))))
    for a, b in (("state", "out"), ("out", "state"), ("out", "q"), ("out", "v"), ("state", "k")):
        assert la_decode(lib, suf, **{**dec, a: dec[b] + 16}) == E.DP_EINVAL, (a, b)
    nf = dict(zip(("x", "w", "b", "z", "y"), map(at, range(5))))
    for b in ("x", "w", "b", "z"):
        assert norm(lib, suf, **{**nf, "y": nf[b] + 16}) == E.DP_EINVAL, b
    assert norm(lib, suf, **{**nf, "y": nf["z"]}) == E.DP_EINVAL
    nb = dict(zip(("x", "dy", "w", "b", "z", "dx", "dw", "db", "dz", "ws"), map(at, range(10))))
    for a, b in (("dx", "dy"), ("dx", "x"), ("dz", "z"), ("dw", "w"), ("dw", "db"), ("dx", "dz"), ("dz", "dy")):
        assert norm_bwd(lib, suf, **{**nb, a: nb[b] + 16}) == E.DP_EINVAL, (a, b)
    assert norm_bwd(lib, suf, **{**nb, "ws": nb["dx"] + 256}) == E.DP_EINVAL


@pytest.mark.parametrize("suf", ["f32", "bf16"])
def test_sizes_past_a_launch_are_refused(lib, suf):
    """A launch has less than 2^32 threads."""
    for kw in (dict(B=2 ** 23, H=2, Hk=2, L=1), dict(B=2 ** 23, H=2, Hk=2, L=1, cu=P), dict(H=65536, Hk=1)):
        assert la_fwd(lib, suf, **kw) == E.DP_ENOTSUP
        assert la_bwd(lib, suf, **kw) == E.DP_ENOTSUP
    assert la_decode(lib, suf, B=2 ** 24, H=1, Hk=1, n=2 ** 24) == E.DP_ENOTSUP
    assert la_decode(lib, suf, H=65536, Hk=1) == E.DP_ENOTSUP
    for fn in (norm, norm_bwd):
        assert fn(lib, suf, rows=1, G=2 ** 18 - 4, D=2048) == E.DP_ENOTSUP
        assert fn(lib, suf, rows=1, G=2 ** 18, D=1) == E.DP_ENOTSUP
    assert copy(lib, [0], [1], page=2 ** 34 + 16) == E.DP_ENOTSUP
    assert copy(lib, [0], [1], page=2 ** 34, nslots=2 ** 20, layers=8) == E.DP_ENOTSUP


def norm(lib, suf, x=P, w=P, b=P, z=None, rows=4, G=2, D=64, eps=1e-5, y=P, flags=0):
    return getattr(lib, f"dp_group_norm_{suf}")(x, w, b, z, rows, G, D, eps, y, flags, None)


def norm_bwd(lib, suf, x=P, dy=P, w=P, b=P, z=None, rows=4, G=2, D=64, eps=1e-5, dx=P, dw=P, db=P, dz=None, ws=P, wsb=BIG,
             flags=0):
    return getattr(lib, f"dp_group_norm_bwd_{suf}")(x, dy, w, b, z, rows, G, D, eps, dx, dw, db, dz, ws, wsb, flags, None)


@pytest.mark.parametrize("suf", ["f32", "bf16"])
def test_norm_checks(lib, suf):
    for fn in (norm, norm_bwd):
        for kw, code in [(dict(rows=-1), E.DP_EINVAL), (dict(G=0), E.DP_EINVAL), (dict(D=0), E.DP_EINVAL),
                         (dict(D=2049), E.DP_ENOTSUP), (dict(eps=-1.0), E.DP_EINVAL), (dict(eps=float("nan")), E.DP_EINVAL),
                         (dict(flags=4), E.DP_EINVAL), (dict(x=None), E.DP_EINVAL), (dict(x=P + 2), E.DP_EINVAL),
                         (dict(rows=2 ** 31), E.DP_ENOTSUP), (dict(w=P + 2), E.DP_EINVAL)]:
            assert fn(lib, suf, **kw) == code, kw
    assert norm(lib, suf, z=P, flags=E.NORM_SILU) == E.DP_EINVAL
    assert norm(lib, suf, y=None) == E.DP_EINVAL
    assert norm(lib, suf, rows=0, x=None, y=None) == E.DP_OK
    assert norm_bwd(lib, suf, z=P) == E.DP_EINVAL      # a gate without its gradient
    assert norm_bwd(lib, suf, dz=P) == E.DP_EINVAL     # and the other way round
    assert norm_bwd(lib, suf, dy=None) == E.DP_EINVAL
    assert norm_bwd(lib, suf, dx=None) == E.DP_EINVAL
    assert norm_bwd(lib, suf, ws=None) == E.DP_EWORKSPACE
    assert norm_bwd(lib, suf, wsb=8) == E.DP_EWORKSPACE
    assert norm_bwd(lib, suf, ws=P + 64) == E.DP_EWORKSPACE
    out = ctypes.c_size_t(0)
    assert lib.dp_group_norm_bwd_workspace_size(4, 2, 64, 3, ctypes.byref(out)) == E.DP_EINVAL
    assert lib.dp_group_norm_bwd_workspace_size(0, 2, 64, 2, ctypes.byref(out)) == E.DP_OK and out.value == 0


def copy(lib, src, dst, pool=P, page=64, nslots=8, layers=2, n=None):
    a, b = (ctypes.c_int * max(1, len(src)))(*src), (ctypes.c_int * max(1, len(dst)))(*dst)
    return lib.dp_state_copy(pool, page, nslots, layers, a, b, len(src) if n is None else n, None)


def test_copy_checks(lib):
    assert copy(lib, [], []) == E.DP_OK
    for src, dst in [([8], [0]), ([-2], [0]), ([0], [8]), ([0], [-1]), ([0, 1], [2, 2]), ([0, 2], [2, 3]), ([3], [3]),
                     ([-1, -1], [4, 4])]:
        assert copy(lib, src, dst) == E.DP_EINVAL, (src, dst)
    assert copy(lib, [0], [1], pool=None) == E.DP_EINVAL
    assert copy(lib, [0], [1], pool=P + 4) == E.DP_EINVAL
    assert copy(lib, [0], [1], page=0) == E.DP_EINVAL
    assert copy(lib, [0], [1], page=6) == E.DP_ENOTSUP
    assert copy(lib, [0], [1], layers=0) == E.DP_EINVAL
    assert copy(lib, [0], [1], layers=65536) == E.DP_ENOTSUP
    assert copy(lib, [0], [1], n=-1) == E.DP_EINVAL
    assert copy(lib, [0] * 9, list(range(9))) == E.DP_EINVAL
    assert lib.dp_state_copy(P, 64, 8, 2, None, None, 1, None) == E.DP_EINVAL


def test_binding_refuses_before_the_library():
    """Shapes, types, strides and devices are checked on the tensors."""
    q, v = torch.zeros(1, 5, 2, 16), torch.zeros(1, 5, 4, 16)
    with pytest.raises(ValueError):
        dp.la_fwd(q, q, v)  # CPU tensors
    with pytest.raises(ValueError):
        dp.la_fwd(q[0], q[0], v)
    with pytest.raises(TypeError):
        dp.la_fwd(q, q.bfloat16(), v)
    with pytest.raises(ValueError):
        dp.la_fwd(q.transpose(1, 2), q.transpose(1, 2), v.transpose(1, 2))
    with pytest.raises(TypeError):
        dp.la_fwd(q.half(), q.half(), v.half())
    with pytest.raises(ValueError):
        dp.la_fwd(q, q, v, torch.zeros(1, 5, 2))
    with pytest.raises(TypeError):
        dp.la_fwd(q, q, v, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(TypeError):
        dp.la_fwd(q, q, v, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        dp.la_fwd(q[0], q[0], v[0], cu_seqlens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        dp.la_bwd(q, q, v, v, grads=dict(ld=torch.zeros(4)))  # no decay, no gradient of it
    with pytest.raises(ValueError):
        dp.la_decode(q[0], q[0], v[0], torch.zeros(5, 2, 16, 16))
    with pytest.raises(ValueError):
        dp.group_norm(torch.zeros(3))
    with pytest.raises(ValueError):
        dp.group_norm(torch.zeros(3, 2, 4), gate=torch.zeros(3, 2, 4), silu=True)
    with pytest.raises(ValueError):
        dp.group_norm(torch.zeros(3, 2, 4), weight=torch.zeros(4))
    with pytest.raises(ValueError):
        dp.group_norm_bwd(torch.zeros(3, 2, 4), torch.zeros(3, 2, 4), grads=dict(gate=torch.zeros(3, 2, 4)))
    with pytest.raises(ValueError):
        dp.state_copy(torch.zeros(2, 3, 4), [0], [1, 2])
    with pytest.raises(ValueError):
        dp.state_copy(torch.zeros(3, 4), [0], [1])
    with pytest.raises(ValueError):
        dp.StatePool(0, 1, 1, 16, 16, device="cpu")


def test_binding_refuses_slots_and_streams(monkeypatch):
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream"):
        binding._On(torch.device("cuda", 0), Stream())
    pool = torch.zeros(2, 3, 4)
    for src, dst in (([2 ** 32], [1]), ([0], [2 ** 32 + 1]), ([3], [1]), ([0], [3])):
        with pytest.raises(ValueError, match="outside the pool"):
            dp.state_copy(pool, src, dst)
    monkeypatch.setattr(binding, "state_copy", lambda *a, **k: None)
    with pytest.raises(ValueError, match="wanted"):
        dp.StatePool(1, 3, 1, 16, 16, device="cpu").alloc(-1)


def test_pool_bookkeeping(monkeypatch):
    """Slots, forks and compaction on the host; the copies recorded, not run."""
    calls = []
    monkeypatch.setattr(binding, "state_copy", lambda pool, src, dst, stream=None: calls.append((list(src), list(dst))))
    p = dp.StatePool(2, 6, 1, 16, 16, device="cpu")
    assert p.alloc(3) == [0, 1, 2] and calls[-1] == ([-1] * 3, [0, 1, 2])
    assert p.fork(1, 2) == [3, 4] and calls[-1] == ([1, 1], [3, 4])
    with pytest.raises(RuntimeError):
        p.alloc(2)
    with pytest.raises(ValueError):
        p.fork(5)
    with pytest.raises(ValueError):
        p.free([0, 0])
    with pytest.raises(ValueError):
        p.free([5])
    p.free([0, 2])
    assert p.compact() == {3: 0, 4: 2} and calls[-1] == ([3, 4], [0, 2])
    assert p.free_slots == 3 and p.compact() == {}
    assert p.alloc(3) == [3, 4, 5]
