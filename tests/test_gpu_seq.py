"""The sequence operators on the GPU against the 64-bit definitions
(tests/seq_reference.py), through the binding's classes.

Tolerances (u = 2^-24, HALF the storage type's half step, relative):

convolution  z is K + 1 fp32 terms: off by (K + 1) u s, s the sum of the terms'
  magnitudes.  |silu'| <= 1.1.  exp(-z) as exp2 of a rounded product is off by
  (|z| + 4) u relative, the division and product by 4 u more; the slope adds z
  times that.  So |y - ref| <= HALF |ref| + (1.1 (K + 1) s + (|z| + 8) (1 + |z|)) u,
  rounded up below to 2 u (K + 8) (1 + s)^2 (|z| <= s).
delta rule   k has length 1 and 0 <= beta <= 1, so a token's map of the state
  never lengthens it and a rounding made in one chunk is not amplified later.
  Each chunk chains at most 6 sums of up to Dk + 64 products; errors of a sum of
  n products of independent rounding add up to sqrt(n) u of its size, twice that
  for the triangular inverse.  2-norms: HALF + 12 sqrt(Dk + 64) u forward, twice
  as many chained sums (the forward pass again, then back) backward.  Elements:
  HALF |ref| + 4 (Dk + 64) u times the largest norm of a state or value times
  the scale (a state element is at most its norm, |q| is the scale).
norms        sums of D squares and products in fp32 and eight more operations an
  element: elements within HALF |ref| + (D + 64) u times the row's largest value
  and 2-norms within HALF + 8 sqrt(D) u.  Sums over rows the same with rows in
  place of D.
"""
import math

import numpy as np
import pytest
import torch

import depthwise_convolution_amd as dw
import seq_reference as ref
from gpu_helpers import DEV, say
from seq_reference import DTYPES, HALF, U, leaves, rel, starts

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0, dtype="f32", std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(1000 * seed + sum((i + 3) * n for i, n in enumerate(shape)))
    return (torch.randn(shape, generator=g) * std + mean).to(DTYPES[dtype])


def offsets_of(lens):
    return torch.tensor(starts(lens), dtype=torch.int32, device=DEV)


def up(t):
    return None if t is None else t.to(DEV)


def strided(t, extra, offset=0):
    """The same values as a slice of wider tokens, `offset` elements in."""
    n = t.shape[0]
    wide = torch.zeros(n, t[0].numel() + extra, dtype=t.dtype, device=t.device)
    view = wide[:, offset:offset + t[0].numel()]
    view.copy_(t.reshape(n, -1))
    return view.unflatten(1, tuple(t.shape[1:])) if t.dim() > 2 else view


def close(got, want, tol, what):
    got = got.detach().double().cpu()
    want = want.detach()
    assert got.shape == want.shape, what
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((got - want).abs().max())}"


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------
def conv_data(fmt, C, K, lens, state, seed=0):
    T = sum(lens)
    return (rand(T, C, seed=seed, dtype=fmt), rand(K, C, seed=seed + 1, dtype=fmt, std=K ** -0.5),
            rand(C, seed=seed + 2, std=0.3), rand(len(lens), K - 1, C, seed=seed + 3, dtype=fmt) if state else None)


def conv_tol(half, want, K, s):
    return half * want.abs() + 2 * U * (K + 8) * (1 + s) ** 2


CONV = [  # fmt, C, K, lens, act, state, extra channels of a wider token, offset in it
    ("bf16", 96, 4, [1], "silu", False, 0, 0),
    ("f32", 130, 2, [64, 65, 1], "silu", True, 0, 0),
    ("f16", 61, 3, [5, 0, 2, 17], "silu", True, 0, 0),
    ("bf16", 128, 8, [200, 3], "none", True, 0, 0),
    ("f32", 7, 5, [0, 0, 9], "silu", False, 0, 0),
    ("bf16", 64, 4, [33, 31, 2, 1, 70], "silu", True, 32, 8),
    ("f16", 64, 6, [130], "silu", False, 5, 3),
    ("f32", 1024, 4, [300, 1, 2, 3, 400], "silu", True, 0, 0),
    ("bf16", 1, 7, [40, 6], "silu", True, 0, 0),
    ("f16", 72, 4, [1, 2, 0, 3, 1] * 40, "silu", True, 0, 0),
    ("bf16", 8, 3, [5000], "silu", False, 0, 0),
]


@pytest.mark.parametrize("case", CONV, ids=lambda c: f"{c[0]}-C{c[1]}-K{c[2]}-{sum(c[3])}")
def test_conv_forward(case):
    fmt, C, K, lens, act, state, extra, off = case
    say(f"[gpu] causal fwd {case}")
    x, w, b, s = conv_data(fmt, C, K, lens, state)
    T, tail = sum(lens), 5
    plan = dw.CausalDepthwiseConv1d(C, K, fmt, act=act)
    xd = up(torch.cat([x, torch.full((tail, C), float("nan"), dtype=x.dtype)]))  # behind the last sequence
    xd = strided(xd, extra, off) if extra else xd
    y = torch.full((T + tail, C), 7.0, dtype=x.dtype, device=DEV)
    so = torch.full((len(lens), K - 1, C), float("nan"), dtype=x.dtype, device=DEV)
    plan(xd, up(w), up(b), offsets=offsets_of(lens), state_in=up(s), state_out=so, y=y)
    want, states, z, sc = ref.conv(x.double(), w.double(), b.double(), lens, None if s is None else s.double(), act)
    close(y[:T], want, conv_tol(HALF[x.dtype], want, K, sc), "y")
    assert (y[T:] == 7.0).all(), "written behind the last sequence"
    assert torch.equal(so.double().cpu(), states)  # copies


@pytest.mark.parametrize("case", CONV, ids=lambda c: f"{c[0]}-C{c[1]}-K{c[2]}-{sum(c[3])}")
def test_conv_backward(case):
    fmt, C, K, lens, act, state, extra, off = case
    say(f"[gpu] causal bwd {case}")
    x, w, b, s = conv_data(fmt, C, K, lens, state, seed=5)
    T, tail = sum(lens), 3
    dy = rand(T, C, seed=11, dtype=fmt)
    dso = rand(len(lens), K - 1, C, seed=12, dtype=fmt) if state else None
    pad = lambda t: up(torch.cat([t, torch.full((tail, C), float("nan"), dtype=t.dtype)]))  # noqa: E731
    xd, dyd = pad(x), pad(dy)
    if extra:
        xd, dyd = strided(xd, extra, off), strided(dyd, extra + 8, off)
    dx = torch.full((T + tail, C), 7.0, dtype=x.dtype, device=DEV)
    plan = dw.CausalDepthwiseConv1d(C, K, fmt, act=act)
    _, dw_, db, ds = plan.backward(xd, up(w), dyd, up(b), offsets=offsets_of(lens), state_in=up(s), dstate_out=up(dso),
                                   dx=dx)
    xs, ws, bs, ss = leaves(x, w, b, s)
    y, st, z, sc = ref.conv(xs, ws, bs, lens, ss, act)
    outs, gives, wrt = [y], [dy.double()], [xs, ws, bs] + ([ss] if state else [])
    if state:
        outs, gives = outs + [st], gives + [dso.double()]
    g = torch.autograd.grad(outs, wrt, gives, allow_unused=True)
    g = [torch.zeros_like(t) if v is None else v for v, t in zip(g, wrt)]
    # a dz is off by its share of z's error times |silu''| <= 0.5, and by the
    # exponential's; dx adds K of them, dw and dbias all tokens' (2-norms)
    top = 1 + float(sc.max()) if T else 1.0
    e = 2 * U * (K + 8) * top ** 2 * (float(dy.abs().max()) if T else 0.0) * K
    close(dx[:T], g[0], HALF[x.dtype] * g[0].abs() + e, "dx")
    assert (dx[T:] == 7.0).all(), "written behind the last sequence"
    many = math.sqrt(max(T, 1)) * e * 4 + U * 64 * max(T, 1) ** 0.5 * top
    close(dw_, g[1], many + 4 * U * g[1].abs(), "dw")
    close(db, g[2], many + 4 * U * g[2].abs(), "dbias")
    if state:
        close(ds, g[3], HALF[x.dtype] * g[3].abs() + e, "dstate")
    else:
        assert ds is None


# wide enough for runs of 64 tokens, in vectors and in single elements
@pytest.mark.parametrize("case", [("f32", 8000, 5, [1500, 690, 1, 9], "silu", True, 0, 0),
                                  ("bf16", 4001, 3, [1100, 0, 1030, 70], "silu", True, 0, 0)],
                         ids=lambda c: f"{c[0]}-C{c[1]}-K{c[2]}")
def test_conv_of_long_runs(case):
    test_conv_forward(case)
    test_conv_backward(case)


def test_conv_one_sequence_without_offsets_and_no_tokens():
    x, w, b, _ = conv_data("f16", 32, 4, [50], False)
    plan = dw.CausalDepthwiseConv1d(32, 4, "f16", act="none")
    one = plan(up(x), up(w))
    two = plan(up(x), up(w), offsets=offsets_of([50]))
    assert torch.equal(one, two)
    s = rand(3, 3, 32, dtype="f16")
    so = torch.empty_like(s, device=DEV)
    empty = torch.empty(0, 32, dtype=torch.float16, device=DEV)
    y = plan(empty, up(w), offsets=offsets_of([0, 0, 0]), state_in=up(s), state_out=so)
    assert y.shape == (0, 32) and torch.equal(so.cpu(), s)
    dx, dw_, db, ds = plan.backward(empty, up(w), empty, up(b), offsets=offsets_of([0, 0, 0]), state_in=up(s),
                                    dstate_out=up(s))
    assert dx.shape == (0, 32) and not dw_.any() and not db.any() and torch.equal(ds.cpu(), s)


@pytest.mark.parametrize("fmt,C,K,rows,act", [("bf16", 96, 4, 5, "silu"), ("f32", 33, 3, 1, "none"),
                                              ("f16", 2050, 2, 70, "silu"), ("bf16", 64, 8, 3, "silu")])
def test_conv_steps_are_the_forward_pass(fmt, C, K, rows, act):
    """Tokens one by one through a cache (slots in any order, one row skipped)
    give the packed pass's values and states."""
    n = 6
    x, w, b, s = conv_data(fmt, C, K, [n] * rows, True)
    plan = dw.CausalDepthwiseConv1d(C, K, fmt, act=act)
    want_state = torch.empty_like(s, device=DEV)
    want = plan(up(x), up(w), up(b), offsets=offsets_of([n] * rows), state_in=up(s), state_out=want_state)
    order = torch.randperm(rows + 2, generator=torch.Generator().manual_seed(3))
    cache = torch.full((rows + 2, K - 1, C), 3.0, dtype=s.dtype, device=DEV)
    cache[order[:rows].to(DEV)] = up(s)
    slots = torch.cat([order[:rows], torch.tensor([-1, rows + 2])]).to(torch.int32).to(DEV)
    for t in range(n):
        xt = torch.cat([up(x)[t::n], torch.full((2, C), float("nan"), dtype=x.dtype, device=DEV)])
        y = torch.full((rows + 2, C), 9.0, dtype=x.dtype, device=DEV)
        plan.step(xt, up(w), up(b), state=cache, slots=slots, y=y)
        assert torch.equal(y[:rows], want[t::n]), f"token {t}"
        assert (y[rows:] == 9.0).all()
    assert torch.equal(cache[order[:rows].to(DEV)], want_state)
    assert (cache[order[rows:].to(DEV)] == 3.0).all()


def test_conv_step_same_slot_twice_and_no_slots():
    """Rows of one slot are consecutive tokens, whatever lies between them."""
    C, K = 40, 4
    x, w, b, s = conv_data("f32", C, K, [7], True)
    plan = dw.CausalDepthwiseConv1d(C, K, "f32")
    cache, rowwise = up(s).repeat(3, 1, 1), up(s).repeat(3, 1, 1)
    slots = torch.tensor([2, 0, 2, 2, 1, 0, 2], dtype=torch.int32, device=DEV)
    y = plan.step(up(x), up(w), up(b), state=cache, slots=slots)
    for i in range(7):
        one = plan.step(up(x)[i:i + 1], up(w), up(b), state=rowwise, slots=slots[i:i + 1])
        assert torch.equal(one[0], y[i])
    assert torch.equal(cache, rowwise)
    a, c = up(s).repeat(3, 1, 1), up(s).repeat(3, 1, 1)
    y0 = plan.step(up(x)[:3], up(w), up(b), state=a)
    y1 = plan.step(up(x)[:3], up(w), up(b), state=c, slots=torch.arange(3, dtype=torch.int32, device=DEV))
    assert torch.equal(y0, y1) and torch.equal(a, c)


def test_wrong_offsets_stay_in_bounds():
    """Offsets that fall or run past the tokens are clamped: outputs outside
    the buffers' guards stay untouched."""
    C, K, T = 32, 4, 40
    x, w, b, _ = conv_data("f32", C, K, [T], False)
    plan = dw.CausalDepthwiseConv1d(C, K, "f32")
    rule = dw.GatedDeltaRule(1, 1, 16, 16, "f32")
    q = up(rand(T, 1, 16, seed=1))
    g, beta = -up(rand(T, 1, seed=2)).abs(), torch.sigmoid(up(rand(T, 1, seed=3)))
    for bad in ([0, 500, 20], [-7, 10, 2 ** 30], [30, 20, 10], [0, 40, -1]):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        buf = torch.full((T + 64, C), 5.0, device=DEV)
        so = torch.empty(2, K - 1, C, device=DEV)
        plan(up(x), up(w), up(b), offsets=off, state_out=so, y=buf[32:32 + T])
        plan.backward(up(x), up(w), up(x), up(b), offsets=off, dx=buf[32:32 + T])
        assert (buf[:32] == 5.0).all() and (buf[32 + T:] == 5.0).all()
        buf = torch.full((T + 64, 1, 16), 5.0, device=DEV)
        rule(q, q, q, g, beta, offsets=off, o=buf[32:32 + T])
        rule.backward(q, q, q, g, beta, q, offsets=off, dq=buf[32:32 + T])
        torch.cuda.synchronize()
        assert (buf[:32] == 5.0).all() and (buf[32 + T:] == 5.0).all()


# ---------------------------------------------------------------------------
# gated delta rule
# ---------------------------------------------------------------------------
def delta_data(fmt, Hk, Hv, Dk, Dv, lens, state, gates="mixed", normalize=True, seed=0):
    T = sum(lens)
    q, k = rand(T, Hk, Dk, seed=seed, dtype=fmt, mean=0.2), rand(T, Hk, Dk, seed=seed + 1, dtype=fmt, mean=0.2)
    if not normalize:  # keys no longer than 1, as the tolerances ask
        k = (k.float() / (1.1 * k.float().norm(dim=-1, keepdim=True).clamp_min(1e-3))).to(DTYPES[fmt])
    v = rand(T, Hv, Dv, seed=seed + 2, dtype=fmt)
    g = -rand(T, Hv, seed=seed + 3).abs() * 0.3
    beta = torch.sigmoid(rand(T, Hv, seed=seed + 4))
    if gates == "mixed" and T:
        g[::7] = 0.0
        g[5::11] = -math.inf      # everything is forgotten
        g[3::17] = -90.0
        beta[::5] = 0.0
        beta[2::6] = 1.0
        k[1::9] = 0.0             # no key at all
    s = rand(len(lens), Hv, Dk, Dv, seed=seed + 5, std=0.3) if state else None
    return q, k, v, g, beta, s


DELTA = [  # fmt, Hk, Hv, Dk, Dv, lens, state, gates, normalize
    ("f32", 1, 1, 16, 16, [1], False, "mixed", True),
    ("f32", 1, 2, 64, 64, [64], True, "plain", True),
    ("f32", 2, 2, 33, 7, [63, 0, 1, 65], True, "mixed", True),
    ("bf16", 2, 4, 128, 128, [130, 70], True, "mixed", True),
    ("f16", 1, 3, 96, 104, [200], False, "plain", True),
    ("bf16", 1, 1, 200, 130, [100, 3], True, "mixed", True),
    ("f16", 1, 1, 256, 80, [97], True, "mixed", True),
    ("f32", 1, 1, 7, 300, [66], True, "plain", True),
    ("bf16", 3, 3, 64, 1, [128, 129], False, "mixed", True),
    ("f32", 1, 1, 1, 2, [70], True, "plain", False),
    ("f16", 2, 2, 64, 48, [80, 5], True, "plain", False),
    ("bf16", 1, 6, 64, 40, [65, 2], True, "mixed", True),      # more value heads than wavefronts
    ("f32", 1, 5, 40, 24, [67], True, "mixed", True),
    ("bf16", 2, 18, 32, 20, [130], False, "plain", True),
    ("f16", 1, 2, 130, 300, [64, 64], True, "mixed", True),
    ("bf16", 1, 2, 24, 33, [1, 2, 0, 3] * 12, True, "mixed", True),
    ("f32", 1, 1, 256, 70, [65], True, "plain", True),
]
IDS = [f"{c[0]}-{c[1]}x{c[2]}-{c[3]}x{c[4]}-{'+'.join(map(str, c[5][:4]))}" for c in DELTA]


def delta_check(got, want, half, n, size, what, chain=1):
    close(got, want, half * want.detach().abs() + 4 * chain * n * U * size, what)
    assert rel(got.cpu(), want.detach()) <= half + 12 * chain * math.sqrt(n) * U, (what, rel(got.cpu(), want.detach()))


@pytest.mark.parametrize("case", DELTA, ids=IDS)
def test_delta_forward(case):
    fmt, Hk, Hv, Dk, Dv, lens, state, gates, norm = case
    say(f"[gpu] delta fwd {case}")
    q, k, v, g, beta, s = delta_data(*case)
    T, tail = sum(lens), 3
    pad = lambda t: up(torch.cat([t, torch.full((tail,) + t.shape[1:], float("nan"), dtype=t.dtype)]))  # noqa: E731
    plan = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, fmt, normalize=norm)
    o = torch.full((T + tail, Hv, Dv), 7.0, dtype=v.dtype, device=DEV)
    so = torch.full((len(lens), Hv, Dk, Dv), float("nan"), device=DEV)
    plan(pad(q), pad(k), pad(v), pad(g), pad(beta), offsets=offsets_of(lens), state_in=up(s), state_out=so, o=o)
    want, states, size = ref.delta(*(t.double() for t in (q, k, v, g, beta)), lens, None if s is None else s.double(),
                                   Dk ** -0.5, norm, 1e-6)
    qlen = 1.0 if norm else float(q.float().norm(dim=-1).max())
    delta_check(o[:T], want, HALF[v.dtype], Dk + 64, size * qlen * Dk ** -0.5, "o")
    delta_check(so, states, HALF[torch.float32], Dk + 64, size, "state")
    assert (o[T:] == 7.0).all(), "written behind the last sequence"


@pytest.mark.parametrize("case", DELTA, ids=IDS)
def test_delta_backward(case):
    fmt, Hk, Hv, Dk, Dv, lens, state, gates, norm = case
    say(f"[gpu] delta bwd {case}")
    q, k, v, g, beta, s = delta_data(*case, seed=40)
    k[1::9] = rand(*k[1::9].shape, seed=77, dtype=fmt, std=0.1)  # a zero key's gradient has no direction
    T, tail = sum(lens), 3
    do = rand(T, Hv, Dv, seed=50, dtype=fmt)
    dso = rand(len(lens), Hv, Dk, Dv, seed=51, std=0.3) if state else None
    pad = lambda t: up(torch.cat([t, torch.full((tail,) + t.shape[1:], float("nan"), dtype=t.dtype)]))  # noqa: E731
    plan = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, fmt, normalize=norm)
    dqb = torch.full((T + tail, Hk, Dk), 7.0, dtype=q.dtype, device=DEV)
    dvb = torch.full((T + tail, Hv, Dv), 7.0, dtype=q.dtype, device=DEV)
    dgb = torch.full((T + tail, Hv), 7.0, device=DEV)
    dq, dk, dv, dg, dbeta, ds = plan.backward(pad(q), pad(k), pad(v), pad(g), pad(beta), pad(do),
                                              offsets=offsets_of(lens), state_in=up(s), dstate_out=up(dso), dq=dqb,
                                              dv=dvb, dg=dgb)
    for t in (dq, dv, dg):
        assert (t[T:] == 7.0).all(), "written behind the last sequence"
    args = leaves(q, k, v, g, beta, s)
    o, states, size = ref.delta(*args[:5], lens, args[5], Dk ** -0.5, norm, 1e-6)
    outs, gives, wrt = [o], [do.double()], args[:5] + ([args[5]] if state else [])
    if state:
        outs, gives = outs + [states], gives + [dso.double()]
    want = list(torch.autograd.grad(outs, wrt, gives))
    # d(-inf)/dg: the state behind it does not depend on g
    want[3] = torch.where(torch.isinf(g), torch.zeros_like(want[3]), want[3])
    half = HALF[q.dtype]
    for name, got, w, h in (("dq", dq, want[0], half), ("dk", dk, want[1], half), ("dv", dv, want[2], half),
                            ("dg", dg, want[3], HALF[torch.float32]), ("dbeta", dbeta, want[4], HALF[torch.float32])):
        top = float(w.abs().max()) + size
        delta_check(got[:T], w, h, Dk + 64 + (Dv if name in ("dq", "dk", "dg", "dbeta") else 0), top, name, chain=2)
    if state:
        delta_check(ds, want[5], HALF[torch.float32], Dk + 64, float(want[5].abs().max()) + size, "dstate", chain=2)
    else:
        assert ds is None


# Heads x sequences x columns enough for the walks of 32 columns (more than 256 of
# them), at every padded key size; the last walk of a head has few columns.
MANY = [(fmt, 1, 3, Dk, 70, [1, 66, 0, 130, 64] * 6, True, gates, True)
        for fmt, Dk, gates in [("bf16", 40, "mixed"), ("bf16", 128, "plain"), ("bf16", 192, "mixed"), ("bf16", 250, "plain"),
                               ("f16", 64, "plain"), ("f16", 100, "mixed"), ("f16", 130, "plain"), ("f16", 256, "mixed")]]
MANY += [("bf16", 2, 8, 96, 33, [65] * 17, False, "mixed", True), ("f32", 1, 3, 72, 70, [1, 66, 0, 130] * 6, True, "mixed", True)]


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}-{c[3]}x{c[4]}-{len(c[5])}")
def test_delta_of_many_sequences(case):
    test_delta_forward(case)
    test_delta_backward(case)


def test_delta_gradient_matches_differences():
    """The kernels' gradient along a direction against their own forward
    pass's differences (fp32: a step of 2^-8 leaves about 2^-16 of curvature
    and 2^-14 of rounding)."""
    Hk, Hv, Dk, Dv, lens = 1, 2, 32, 32, [70, 20]
    q, k, v, g, beta, s = (up(t) for t in delta_data("f32", Hk, Hv, Dk, Dv, lens, True, gates="plain"))
    plan, off = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, "f32"), offsets_of(lens)
    do, dso = up(rand(90, Hv, Dv, seed=60)), up(rand(2, Hv, Dk, Dv, seed=61))
    grads = plan.backward(q, k, v, g, beta, do, offsets=off, state_in=s, dstate_out=dso)

    def value(*a):
        so = torch.empty_like(s)
        o = plan(*a[:5], offsets=off, state_in=a[5], state_out=so)
        return float((o.double() * do.double()).sum() + (so.double() * dso.double()).sum())

    args = [q, k, v, g, beta, s]
    for i, name in enumerate(("q", "k", "v", "g", "beta", "state")):
        d = up(rand(*args[i].shape, seed=70 + i))
        h = 2.0 ** -8
        hi, lo = ([a + (sign * h * d if j == i else 0) for j, a in enumerate(args)] for sign in (1, -1))
        slope = (value(*hi) - value(*lo)) / (2 * h)
        along = float((grads[i].double() * d.double()).sum())
        spread = float((grads[i].double().abs() * d.double().abs()).sum())
        assert abs(slope - along) <= 2e-3 * spread, (name, slope, along)


def test_delta_takes_slices_of_one_tensor():
    """q, k and v as views of one tensor (odd offsets: unaligned rows) give the
    bits of dense ones, and gradients land in such views."""
    Hk, Hv, Dk, Dv, lens = 2, 4, 32, 32, [100, 29]
    q, k, v, g, beta, _ = delta_data("bf16", Hk, Hv, Dk, Dv, lens, False)
    plan, off = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, "bf16"), offsets_of(lens)
    g, beta, do = up(g), up(beta), up(rand(129, Hv, Dv, seed=9, dtype="bf16"))
    want = plan(up(q), up(k), up(v), g, beta, offsets=off)
    want_g = plan.backward(up(q), up(k), up(v), g, beta, do, offsets=off)
    for lead in (0, 3):
        wide = torch.zeros(129, lead + 2 * Hk * Dk + Hv * Dv, dtype=torch.bfloat16, device=DEV)
        grad = torch.zeros_like(wide)
        cut = lambda t: [x.unflatten(1, s) for x, s in zip(  # noqa: E731
            t[:, lead:].split([Hk * Dk, Hk * Dk, Hv * Dv], 1), ((Hk, Dk), (Hk, Dk), (Hv, Dv)))]
        for view, t in zip(cut(wide), (q, k, v)):
            view.copy_(t)
        assert torch.equal(plan(*cut(wide), g, beta, offsets=off), want)
        dq, dk, dv = cut(grad)
        plan.backward(*cut(wide), g, beta, do, offsets=off, dq=dq, dk=dk, dv=dv)
        for a, b in zip((dq, dk, dv), want_g):
            assert torch.equal(a, b)


STEP = [("f32", 1, 1, 16, 16, 1), ("bf16", 2, 4, 128, 128, 9), ("f16", 1, 2, 96, 50, 5), ("bf16", 1, 1, 256, 33, 3),
        ("f32", 2, 2, 7, 5, 4), ("bf16", 4, 8, 128, 128, 70), ("f16", 1, 1, 200, 64, 600)]


@pytest.mark.parametrize("case", STEP, ids=lambda c: "-".join(map(str, c)))
def test_delta_steps_follow_the_definition(case):
    fmt, Hk, Hv, Dk, Dv, rows = case
    say(f"[gpu] delta step {case}")
    n = 3
    q, k, v, g, beta, s = delta_data(fmt, Hk, Hv, Dk, Dv, [n] * rows, True)
    plan = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, fmt)
    want, states, size = ref.delta(*(t.double() for t in (q, k, v, g, beta)), [n] * rows, s.double(), Dk ** -0.5, True,
                                   1e-6)
    order = torch.randperm(rows + 2, generator=torch.Generator().manual_seed(3))
    cache = torch.full((rows + 2, Hv, Dk, Dv), 3.0, device=DEV)
    cache[order[:rows].to(DEV)] = up(s)
    slots = torch.cat([order[:rows], torch.tensor([-1, rows + 2])]).to(torch.int32).to(DEV)
    tail = lambda t: torch.cat([up(t.contiguous()), torch.full((2,) + t.shape[1:], float("nan"), dtype=t.dtype,  # noqa: E731
                                                               device=DEV)])
    for t in range(n):
        o = torch.full((rows + 2, Hv, Dv), 9.0, dtype=v.dtype, device=DEV)
        plan.step(*(tail(a[t::n]) for a in (q, k, v, g, beta)), state=cache, slots=slots, o=o)
        assert (o[rows:] == 9.0).all()
        delta_check(o[:rows], want[t::n], HALF[v.dtype], Dk + 64, size * Dk ** -0.5, f"o {t}")
    delta_check(cache[order[:rows].to(DEV)], states, HALF[torch.float32], Dk + 64, size, "state")
    assert (cache[order[rows:].to(DEV)] == 3.0).all()


def test_delta_step_same_slot_twice_and_no_slots():
    Hk, Hv, Dk, Dv = 1, 2, 64, 64
    q, k, v, g, beta, s = (up(t) for t in delta_data("bf16", Hk, Hv, Dk, Dv, [7], True))
    plan = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, "bf16")
    cache, rowwise = s.repeat(3, 1, 1, 1), s.repeat(3, 1, 1, 1)
    slots = torch.tensor([2, 0, 2, 2, 1, 0, 2], dtype=torch.int32, device=DEV)
    o = plan.step(q, k, v, g, beta, state=cache, slots=slots)
    for i in range(7):
        one = plan.step(*(t[i:i + 1] for t in (q, k, v, g, beta)), state=rowwise, slots=slots[i:i + 1])
        assert torch.equal(one[0], o[i])
    assert torch.equal(cache, rowwise)
    a, b = s.repeat(3, 1, 1, 1), s.repeat(3, 1, 1, 1)
    first = tuple(t[:3] for t in (q, k, v, g, beta))
    assert torch.equal(plan.step(*first, state=a),
                       plan.step(*first, state=b, slots=torch.arange(3, dtype=torch.int32, device=DEV)))
    assert torch.equal(a, b)


def test_delta_state_in_place_and_no_tokens():
    Hk, Hv, Dk, Dv, lens = 1, 2, 64, 96, [80, 0, 65]
    q, k, v, g, beta, s = (up(t) for t in delta_data("f16", Hk, Hv, Dk, Dv, lens, True))
    plan, off = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, "f16"), offsets_of(lens)
    out = torch.empty_like(s)
    o = plan(q, k, v, g, beta, offsets=off, state_in=s, state_out=out)
    both = s.clone()
    o2 = plan(q, k, v, g, beta, offsets=off, state_in=both, state_out=both)
    assert torch.equal(o, o2) and torch.equal(out, both) and torch.equal(out[1], s[1])
    e = [t[:0] for t in (q, k, v, g, beta)]
    none = offsets_of([0, 0, 0])
    got = torch.empty_like(s)
    assert plan(*e, offsets=none, state_in=s, state_out=got).shape == (0, Hv, Dv) and torch.equal(got, s)
    grads = plan.backward(*e, v[:0], offsets=none, state_in=s, dstate_out=s)
    assert torch.equal(grads[5], s)


def test_caches_past_32_bits():
    """The last entries of caches of more than 2^31 elements."""
    rule = dw.GatedDeltaRule(1, 2, 128, 128, "bf16")
    n = 2 ** 31 // (2 * 128 * 128) + 3
    cache = torch.empty(n, 2, 128, 128, device=DEV)
    q, k, v, g, beta, s = (up(t) for t in delta_data("bf16", 1, 2, 128, 128, [2], True))
    small = s.repeat(2, 1, 1, 1)
    cache[n - 2:] = small
    o = rule.step(q, k, v, g, beta, state=cache, slots=torch.tensor([n - 1, n - 2], dtype=torch.int32, device=DEV))
    o2 = rule.step(q, k, v, g, beta, state=small, slots=torch.tensor([1, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(o, o2) and torch.equal(cache[n - 2:], small)
    del cache
    conv = dw.CausalDepthwiseConv1d(8192, 4, "bf16")
    n = 2 ** 31 // (3 * 8192) + 3
    cache = torch.empty(n, 3, 8192, dtype=torch.bfloat16, device=DEV)
    x, w, b, s = (up(t) for t in conv_data("bf16", 8192, 4, [2], True))
    small = s.repeat(2, 1, 1)
    cache[n - 2:] = small
    y = conv.step(x, w, b, state=cache, slots=torch.tensor([n - 1, n - 2], dtype=torch.int32, device=DEV))
    y2 = conv.step(x, w, b, state=small, slots=torch.tensor([1, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(y, y2) and torch.equal(cache[n - 2:], small)
    del cache
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# norms around a block
# ---------------------------------------------------------------------------
NORM = [  # fmt, rows, D, after, before, act, per (0: no gate), residual, scale
    ("bf16", 37, 128, "rms", "none", "silu", 1, False, False),
    ("f16", 49, 96, "layer", "layer", "sigmoid", 7, True, True),
    ("f32", 5, 1, "rms", "rms", "none", 0, True, True),
    ("f32", 33, 61, "layer", "rms", "silu", 4, True, False),
    ("bf16", 20, 512, "none", "rms", "none", 0, True, True),
    ("f16", 9, 520, "rms", "layer", "none", 1, False, True),
    ("bf16", 7, 2048, "rms", "rms", "silu", 3, True, True),
    ("f32", 6, 4096, "rms", "rms", "none", 0, True, True),
    ("bf16", 3, 8200, "layer", "none", "sigmoid", 1, True, False),
    ("f16", 2, 16383, "rms", "layer", "silu", 2, True, True),
    ("bf16", 4100, 64, "rms", "layer", "sigmoid", 1, True, True),
    ("f32", 5000, 40, "layer", "rms", "silu", 2, True, True),
    ("f16", 3000, 128, "rms", "none", "sigmoid", 1500, False, True),
    ("bf16", 1, 4096, "rms", "rms", "none", 0, True, False),
]
NIDS = [f"{c[0]}-{c[1]}x{c[2]}-{c[3]}-{c[4]}-{c[5]}{c[6]}" for c in NORM]
PARAMS = ("residual", "gate", "scale", "w_after", "b_after", "w_before", "b_before")


def norm_data(case, seed=0):
    fmt, rows, D, after, before, act, per, residual, scale = case
    d = {"o": rand(rows, D, seed=seed, dtype=fmt, mean=0.3)}
    d["residual"] = rand(rows, D, seed=seed + 1, dtype=fmt) if residual else None
    d["gate"] = rand(-(-rows // per), D, seed=seed + 2, dtype=fmt) if per else None
    d["scale"] = rand(D, seed=seed + 3, std=0.2, mean=0.5) if scale else None
    for i, (side, kind) in enumerate((("after", after), ("before", before))):
        d["w_" + side] = rand(D, seed=seed + 4 + i, std=0.2, mean=1.0) if kind != "none" else None
        d["b_" + side] = rand(D, seed=seed + 6 + i, std=0.2) if kind == "layer" else None
    return d


def norm_ref(case, d):
    fmt, rows, D, after, before, act, per, residual, scale = case
    return ref.block(d["o"], d["residual"], d["gate"], max(per, 1), d["scale"], d["w_after"], d["b_after"],
                     d["w_before"], d["b_before"], after, before, act, 1e-6)


def norm_check(got, want, half, n, what, lift=1.0):
    want = want.detach()
    flat = want.reshape(-1, want.shape[-1]) if want.dim() > 1 else want[None]
    top = flat.abs().amax(1, keepdim=True).expand_as(flat).reshape(want.shape)
    close(got, want, half * want.abs() + (n + 64) * U * (top + lift), what)
    r = rel(got.cpu(), want)
    assert r <= half + 8 * math.sqrt(n + 64) * U * max(1.0, lift), (what, r)


@pytest.mark.parametrize("case", NORM, ids=NIDS)
def test_norm_forward(case):
    fmt, rows, D, after, before, act, per, residual, scale = case
    say(f"[gpu] norm fwd {case}")
    d = norm_data(case)
    plan = dw.BlockNorm(D, fmt, after=after, before=before, gate_act=act)
    args = {n: up(d[n]) for n in PARAMS}
    guard = torch.full((rows + 2, D), 7.0, dtype=d["o"].dtype, device=DEV)
    h, y = plan(up(d["o"]), rows_per_gate=max(per, 1), h=guard[1:rows + 1] if D % 8 == 0 else None, **args)
    assert (guard[0] == 7.0).all() and (guard[-1] == 7.0).all()
    want_h, want_y = norm_ref(case, {n: None if t is None else t.double() for n, t in d.items()})
    norm_check(h, want_h, HALF[h.dtype], D, "h")
    if before == "none":
        assert y is None
    else:
        norm_check(y, want_y, HALF[h.dtype], D, "y")


@pytest.mark.parametrize("case", [c for c in NORM if c[2] > 1], ids=[i for i, c in zip(NIDS, NORM) if c[2] > 1])
def test_norm_backward(case):
    fmt, rows, D, after, before, act, per, residual, scale = case
    say(f"[gpu] norm bwd {case}")
    d = norm_data(case, seed=20)
    dh, dy = rand(rows, D, seed=30, dtype=fmt), rand(rows, D, seed=31, dtype=fmt)
    plan = dw.BlockNorm(D, fmt, after=after, before=before, gate_act=act)
    got = plan.backward(up(d["o"]), up(dh), up(dy) if before != "none" else None, rows_per_gate=max(per, 1),
                        **{n: up(d[n]) for n in PARAMS})
    names = ("o",) + PARAMS
    lv = dict(zip(names, leaves(*(d[n] for n in names))))
    h, y = norm_ref(case, lv)
    outs, gives = ([h], [dh.double()]) if y is None else ([h, y], [dh.double(), dy.double()])
    have = [n for n in names if lv[n] is not None]
    want = dict(zip(have, torch.autograd.grad(outs, [lv[n] for n in have], gives)))
    # 1 / |row| of either norm can lift an error: by its largest value
    lift = 1.0
    for x, kind in ((lv["o"].detach(), after), (h.detach(), before)):
        if kind != "none":
            c = x - x.mean(-1, keepdim=True) if kind == "layer" else x
            lift *= max(1.0, float((c.square().mean(-1) + 1e-6).rsqrt().max()))
    for n, g in zip(names, got):
        if n not in want:
            assert g is None, n
            continue
        summed = n in ("scale", "w_after", "b_after", "w_before", "b_before") or (n == "gate" and per > 1)
        norm_check(g, want[n], HALF[g.dtype], D + (rows if summed else 0), n, lift=lift)


def test_norm_in_place_and_unwanted_gradients():
    case = ("bf16", 21, 256, "rms", "rms", "silu", 1, True, True)
    d = {n: up(t) for n, t in norm_data(case).items()}
    plan = dw.BlockNorm(256, "bf16")
    args = {n: d[n] for n in PARAMS}
    h, y = plan(d["o"], **args)
    res, o = d["residual"].clone(), d["o"].clone()
    h2, y2 = plan(o, **{**args, "residual": res}, h=res, y=o)
    assert torch.equal(h, h2) and torch.equal(y, y2) and h2 is res and y2 is o
    dy = up(rand(21, 256, seed=3, dtype="bf16"))
    want = plan.backward(d["o"], None, dy, **args)  # dh = 0
    zero = plan.backward(d["o"], torch.zeros_like(dy), dy, **args)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(want, zero))
    # only do, through the C ABI
    ws = torch.empty(dw.dwconv_norm_bwd_workspace(plan.handle, 21, 1), dtype=torch.uint8, device=DEV)
    do = torch.empty_like(dy)
    dw.dwconv_norm_bwd(plan.handle, 21, d["o"], d["residual"], d["gate"], 1, d["scale"], d["w_after"], None,
                       d["w_before"], None, None, dy, do, None, None, None, None, None, None, None, ws,
                       torch.cuda.current_stream().cuda_stream)
    assert torch.equal(do, want[0])
    # no rows
    e = dw.BlockNorm(256, "bf16")
    assert e(d["o"][:0], **{**args, "residual": d["residual"][:0], "gate": d["gate"][:0]})[1].shape == (0, 256)
    grads = e.backward(d["o"][:0], None, dy[:0], **{**args, "residual": d["residual"][:0], "gate": d["gate"][:0]})
    assert grads[3].abs().sum() == 0 and grads[6].abs().sum() == 0


def test_norm_rows_of_zeros_and_infinities():
    """A row of zeros gives zeros; an infinity spoils its own row alone."""
    o = torch.zeros(6, 64, device=DEV)
    o[1] = 1.0
    o[3, 5] = math.inf
    plan = dw.BlockNorm(64, "f32", after="rms", before="layer")
    w = torch.ones(64, device=DEV)
    h, y = plan(o, w_after=w, w_before=w)
    ok = torch.tensor([0, 1, 2, 4, 5], device=DEV)
    assert torch.isfinite(h[ok]).all() and torch.isfinite(y[ok]).all() and (h[0] == 0).all() and (y[2] == 0).all()
    assert torch.isnan(h[3]).any()


@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_norm_of_unaligned_rows_and_large_gate_groups(fmt):
    """Dense tensors that begin one element into their storage give the bits of
    aligned ones where the sums are formed alike (single elements against
    vectors: the same lanes hold other channels, so within rounding), and a gate
    row may serve more rows than there are."""
    D, rows = 192, 50
    case = (fmt, rows, D, "layer", "rms", "silu", 2 ** 31 - 1, True, True)
    d = norm_data(case)
    plan = dw.BlockNorm(D, fmt, after="layer", before="rms")
    dy = rand(rows, D, seed=3, dtype=fmt)

    def shifted(t):
        if t is None:
            return None
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        buf[1:] = t.reshape(-1).to(DEV)
        return buf[1:].view(t.shape)

    out = []
    for move in (up, shifted):
        args = {n: move(d[n]) for n in PARAMS}
        h, y = plan(move(d["o"]), rows_per_gate=2 ** 31 - 1, **args)
        g = plan.backward(move(d["o"]), move(dy), move(dy), rows_per_gate=2 ** 31 - 1, **args)
        out.append([h, y] + list(g))
    for a, b in zip(*out):
        assert (a is None) == (b is None)
        if a is not None:
            assert rel(a.cpu(), b.double().cpu()) <= 2 * HALF[a.dtype] + 1e-5


def test_no_sequences():
    """Offsets of no sequence at all: nothing is written but sums of nothing."""
    off = torch.zeros(1, dtype=torch.int32, device=DEV)
    T, C = 130, 32
    x, w, b, _ = (up(t) for t in conv_data("bf16", C, 4, [T], False))
    conv = dw.CausalDepthwiseConv1d(C, 4, "bf16")
    y = torch.full((T, C), 7.0, dtype=torch.bfloat16, device=DEV)
    conv(x, w, b, offsets=off, y=y)
    dx, dw_, db, _ = conv.backward(x, w, x, b, offsets=off, dx=y)
    assert (y == 7.0).all() and not dw_.any() and not db.any()
    for fmt in ("f32", "bf16"):
        q, k, v, g, beta, _ = (up(t) for t in delta_data(fmt, 1, 2, 32, 32, [T], False))
        rule = dw.GatedDeltaRule(1, 2, 32, 32, fmt)
        o = torch.full((T, 2, 32), 7.0, dtype=v.dtype, device=DEV)
        rule(q, k, v, g, beta, offsets=off, o=o)
        rule.backward(q, k, v, g, beta, v, offsets=off, dv=o)
        assert (o == 7.0).all()


@pytest.mark.parametrize("fmt,Dk,Dv", [("bf16", 128, 64), ("f16", 64, 64), ("f32", 64, 64)])
def test_long_sequence_in_pieces(fmt, Dk, Dv):
    """A long sequence in one call and in three with the state carried over, at
    borders that no chunk ends on: the same values within fp32 rounding."""
    T, cuts = 6001, [0, 1234, 1235, 6001]
    q, k, v, g, beta, s = (up(t) for t in delta_data(fmt, 1, 2, Dk, Dv, [T], True, gates="plain"))
    g *= 0.05  # slow decay: the state carries far
    rule = dw.GatedDeltaRule(1, 2, Dk, Dv, fmt)
    end, state = torch.empty_like(s), s.clone()
    whole = rule(q, k, v, g, beta, state_in=s, state_out=end)
    parts = [rule(*(t[a:b] for t in (q, k, v, g, beta)), state_in=state, state_out=state) for a, b in zip(cuts, cuts[1:])]
    tol = 24 * math.sqrt(Dk + 64) * U
    assert rel(torch.cat(parts).cpu(), whole.double().cpu()) <= 2 * HALF[v.dtype] + tol
    assert rel(state.cpu(), end.double().cpu()) <= tol


def test_two_streams_at_once():
    """One plan on two streams, a workspace for each call."""
    rule = dw.GatedDeltaRule(2, 4, 64, 64, "bf16")
    sets = [[up(t) for t in delta_data("bf16", 2, 4, 64, 64, [300, 77], True, seed=s)] for s in (0, 100)]
    off = offsets_of([300, 77])
    do = up(rand(377, 4, 64, seed=5, dtype="bf16"))
    want = [rule.backward(*t[:5], do, offsets=off, state_in=t[5]) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for st, t in zip(streams, sets):
            st.wait_stream(torch.cuda.current_stream())
            got.append(rule.backward(*t[:5], do, offsets=off, state_in=t[5], stream=st))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---------------------------------------------------------------------------
# as they are used: a mixer's pass, other streams, captured graphs
# ---------------------------------------------------------------------------
class Mixer:
    """conv -> split -> delta rule -> gated norm of the heads -> residual and the
    next norm, forward and backward, with the operators' classes alone."""

    def __init__(self, fmt, Hk, Hv, D):
        self.Hk, self.Hv, self.D, self.C = Hk, Hv, D, (2 * Hk + Hv) * D
        self.conv = dw.CausalDepthwiseConv1d(self.C, 4, fmt)
        self.rule = dw.GatedDeltaRule(Hk, Hv, D, D, fmt)
        self.heads = dw.BlockNorm(D, fmt, after="rms", before="none")
        self.block = dw.BlockNorm(Hv * D, fmt, after="none", before="rms", gate_act="none")

    def split(self, t):
        q, k, v = t.split([self.Hk * self.D, self.Hk * self.D, self.Hv * self.D], 1)
        return q.unflatten(1, (self.Hk, self.D)), k.unflatten(1, (self.Hk, self.D)), v.unflatten(1, (self.Hv, self.D))

    def forward(self, p, off=None, conv_state=None, conv_out=None, state=None, state_out=None):
        mixed = self.conv(p["x"], p["w"], p["bias"], offsets=off, state_in=conv_state, state_out=conv_out)
        o = self.rule(*self.split(mixed), p["g"], p["beta"], offsets=off, state_in=state, state_out=state_out)
        z, _ = self.heads(o, gate=p["gate"], w_after=p["w_head"])
        h, y = self.block(z.flatten(1), residual=p["res"], scale=p["scale"], w_before=p["w_next"])
        return mixed, o, z, h, y

    def step(self, p, conv_cache, cache, slots):
        mixed = self.conv.step(p["x"], p["w"], p["bias"], state=conv_cache, slots=slots)
        o = self.rule.step(*self.split(mixed), p["g"], p["beta"], state=cache, slots=slots)
        z, _ = self.heads(o, gate=p["gate"], w_after=p["w_head"])
        return self.block(z.flatten(1), residual=p["res"], scale=p["scale"], w_before=p["w_next"])

    def backward(self, p, mixed, o, z, dh, dy, off=None, state=None):
        dz, dres, _, dscale, _, _, dnext, _ = self.block.backward(z.flatten(1), dh, dy, residual=p["res"],
                                                                  scale=p["scale"], w_before=p["w_next"])
        do, _, dgate, _, dhead, _, _, _ = self.heads.backward(o, dz.view_as(o), gate=p["gate"], w_after=p["w_head"])
        dmix = torch.empty_like(mixed)
        dq, dk, dv = self.split(dmix)
        _, _, _, dg, dbeta, ds = self.rule.backward(*self.split(mixed), p["g"], p["beta"], do, offsets=off,
                                                    state_in=state, dq=dq, dk=dk, dv=dv)
        dx, dw_, db, _ = self.conv.backward(p["x"], p["w"], dmix, p["bias"], offsets=off)
        return {"x": dx, "w": dw_, "bias": db, "g": dg, "beta": dbeta, "gate": dgate, "w_head": dhead, "res": dres,
                "scale": dscale, "w_next": dnext, "state": ds}


def mixer_data(m, fmt, T, seed=0):
    p = {"x": rand(T, m.C, seed=seed, dtype=fmt), "w": rand(4, m.C, seed=seed + 1, dtype=fmt, std=0.5),
         "bias": rand(m.C, seed=seed + 2, std=0.1), "g": -rand(T, m.Hv, seed=seed + 3).abs() * 0.2,
         "beta": torch.sigmoid(rand(T, m.Hv, seed=seed + 4)), "gate": rand(T, m.Hv, m.D, seed=seed + 5, dtype=fmt),
         "w_head": rand(m.D, seed=seed + 6, std=0.1, mean=1.0), "res": rand(T, m.Hv * m.D, seed=seed + 7, dtype=fmt),
         "scale": rand(m.Hv * m.D, seed=seed + 8, std=0.1, mean=0.5),
         "w_next": rand(m.Hv * m.D, seed=seed + 9, std=0.1, mean=1.0)}
    return p


def mixer_reference(m, p, lens, state):
    mixed, _, _, _ = ref.conv(p["x"], p["w"], p["bias"], lens, None, "silu")
    q, k, v = m.split(mixed)
    o, S, _ = ref.delta(q, k, v, p["g"], p["beta"], lens, state, m.D ** -0.5, True, 1e-6)
    z, _ = ref.block(o.flatten(0, 1), None, p["gate"].flatten(0, 1), 1, None, p["w_head"], None, None, None, "rms",
                     "none", "silu", 1e-6)
    return ref.block(z.view(o.shape[0], -1), p["res"], None, 1, p["scale"], None, None, p["w_next"], None, "none",
                     "rms", "none", 1e-6)


@pytest.mark.parametrize("fmt", ["f32", "bf16", "f16"])
def test_mixer_forward_and_gradients(fmt):
    """The whole run against the definition in 64 bits.  Four operators round
    to the storage type on the way and as many on the way back: 2-norms within
    16 half steps (each gain below 2) and, for fp32, within 1e-5 as well."""
    m, lens = Mixer(fmt, 1, 2, 64), [90, 41]
    p = mixer_data(m, fmt, 131)
    state = rand(2, 2, 64, 64, seed=30, std=0.2)
    dh, dy = rand(131, 128, seed=31, dtype=fmt), rand(131, 128, seed=32, dtype=fmt)
    off = offsets_of(lens)
    pd = {n: up(t) for n, t in p.items()}
    mixed, o, z, h, y = m.forward(pd, off, state=up(state))
    got = m.backward(pd, mixed, o, z, up(dh), up(dy), off, state=up(state))
    lv = dict(zip(p, leaves(*p.values())))
    s64 = state.double().requires_grad_()
    wh, wy = mixer_reference(m, lv, lens, s64)
    want = dict(zip(list(lv) + ["state"], torch.autograd.grad([wh, wy], list(lv.values()) + [s64],
                                                              [dh.double(), dy.double()])))
    tol = max(16 * HALF[h.dtype], 1e-5)
    for name, a, b in [("h", h, wh), ("y", y, wy)] + [(n, got[n], want[n]) for n in want]:
        r = rel(a.cpu(), b.detach())
        assert r <= tol, (name, r, tol)


def test_mixer_prefill_then_tokens():
    """Prefill of prompts, then tokens through the caches, against one pass
    over all tokens: the same values within the storage type's roundings (the
    chunked and the recurrent form differ by fp32 rounding, which can move a
    rounded value by one step)."""
    fmt, lens, more = "bf16", [70, 9], 5
    m = Mixer(fmt, 2, 2, 64)
    p = mixer_data(m, fmt, sum(lens) + 2 * more)
    rows, a = [], 0
    for n in lens:
        rows.append(list(range(a, a + n + more)))
        a += n + more
    pd = {n: up(t) for n, t in p.items()}
    per_token = ("x", "g", "beta", "gate", "res")
    take = lambda idx: {n: (t[torch.tensor(idx, device=DEV)] if n in per_token else t) for n, t in pd.items()}  # noqa: E731
    whole_off = offsets_of([n + more for n in lens])
    _, _, _, h, y = m.forward(pd, whole_off)
    conv_cache = torch.zeros(4, 3, m.C, dtype=torch.bfloat16, device=DEV)
    cache = torch.zeros(4, 2, 64, 64, device=DEV)
    cs, st = torch.empty(2, 3, m.C, dtype=torch.bfloat16, device=DEV), torch.empty(2, 2, 64, 64, device=DEV)
    pre = [i for r, n in zip(rows, lens) for i in r[:n]]
    _, _, _, hp, yp = m.forward(take(pre), offsets_of(lens), conv_out=cs, state_out=st)
    slots = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    conv_cache[slots.long()], cache[slots.long()] = cs, st
    assert torch.equal(hp, h[torch.tensor(pre, device=DEV)])
    for t in range(more):
        idx = [r[n + t] for r, n in zip(rows, lens)]
        hs, ys = m.step(take(idx), conv_cache, cache, slots)
        sel = torch.tensor(idx, device=DEV)
        assert rel(hs, h[sel].double()) <= 2 * HALF[h.dtype] and rel(ys, y[sel].double()) <= 2 * HALF[h.dtype]


def test_same_bits_again_on_another_stream_and_captured():
    """Every pass gives the same bits on a side stream and in a captured graph
    that is replayed between eager work, its outputs cleared before."""
    fmt, lens = "bf16", [100, 60, 1]
    m = Mixer(fmt, 1, 2, 64)
    pd = {n: up(t) for n, t in mixer_data(m, fmt, 161).items()}
    off, state = offsets_of(lens), up(rand(3, 2, 64, 64, seed=30, std=0.2))
    dh, dy = up(rand(161, 128, seed=31, dtype=fmt)), up(rand(161, 128, seed=32, dtype=fmt))

    def passes():
        mixed, o, z, h, y = m.forward(pd, off, state=state)
        g = m.backward(pd, mixed, o, z, dh, dy, off, state=state)
        return [mixed, o, z, h, y] + [g[n] for n in sorted(g)]

    want = passes()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(passes(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # the argument, as a torch stream and as a raw handle, and the current stream
    y1 = m.conv(pd["x"], pd["w"], pd["bias"], offsets=off, stream=side)
    y2 = m.conv(pd["x"], pd["w"], pd["bias"], offsets=off, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y1, want[0]) and torch.equal(y2, want[0])
    with torch.cuda.stream(side):
        got = passes()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = passes()
    for _ in range(3):
        for t in captured:
            t.fill_(-7)
        eager = passes()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
        assert all(torch.equal(a, b) for a, b in zip(eager, want))
    del graph


def test_captured_steps():
    """A decode step captured once and replayed: caches move on as eagerly."""
    m = Mixer("f16", 1, 2, 64)
    pd = {n: up(t) for n, t in mixer_data(m, "f16", 3).items()}
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device=DEV)
    cc, c = up(rand(3, 3, m.C, seed=1, dtype="f16")), up(rand(3, 2, 64, 64, seed=2))
    mixed, o = torch.zeros(3, m.C, dtype=torch.float16, device=DEV), torch.zeros(3, 2, 64, dtype=torch.float16,
                                                                                  device=DEV)

    def step(conv_cache, cache):
        m.conv.step(pd["x"], pd["w"], pd["bias"], state=conv_cache, slots=slots, y=mixed)
        m.rule.step(*m.split(mixed), pd["g"], pd["beta"], state=cache, slots=slots, o=o)

    ecc, ec = cc.clone(), c.clone()
    step(ecc.clone(), ec.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cc, c)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone()
        step(ecc, ec)
        torch.cuda.synchronize()
        assert torch.equal(got, o) and torch.equal(cc, ecc) and torch.equal(c, ec)
    del graph


def test_binding_refuses():
    """Shapes, types and strides that the kernels do not take."""
    x, w = torch.zeros(4, 8, device=DEV), torch.zeros(4, 8, device=DEV)
    conv = dw.CausalDepthwiseConv1d(8, 4, "f32")
    state = torch.zeros(1, 3, 8, device=DEV)
    for bad in (lambda: conv(x.half(), w), lambda: conv(x[:, :7], w), lambda: conv(x.t(), w), lambda: conv(x, w[:3]),
                lambda: conv(x, w, torch.zeros(7, device=DEV)), lambda: conv(x, w, offsets=torch.tensor([0, 4], device=DEV)),
                lambda: conv(x, w, state_in=state[:, :2]), lambda: conv(x, w, state_in=state.cpu()),
                lambda: conv(x.expand(4, 8)[:1].expand(4, 8), w),
                lambda: conv.step(x, w, None, state=state),
                lambda: conv.step(x, w, None, state=state, slots=torch.zeros(4, dtype=torch.int64, device=DEV)),
                lambda: conv.backward(x, w, x[:3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dw.DwconvError):
        conv(x, w, state_in=state, state_out=state)
    rule = dw.GatedDeltaRule(1, 2, 8, 8, "f32")
    q, v, g = torch.zeros(4, 1, 8, device=DEV), torch.zeros(4, 2, 8, device=DEV), torch.zeros(4, 2, device=DEV)
    small = torch.empty(8, dtype=torch.uint8, device=DEV)
    for bad in (lambda: rule(q, q, q, g, g), lambda: rule(q, q, v, g[:, :1], g), lambda: rule(q, q, v, g.double(), g),
                lambda: rule(q, q, v, g, g, workspace=small), lambda: rule(q, q, v.transpose(1, 2), g, g),
                lambda: rule(q, q, v, g, g, state_out=torch.zeros(1, 2, 8, 8, device=DEV, dtype=torch.float64)),
                lambda: rule.step(q, q, v, g, g, state=torch.zeros(3, 2, 8, 8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    norm = dw.BlockNorm(8, "f32")
    one = torch.ones(8, device=DEV)
    for bad in (lambda: norm(x[:, :4], w_after=one, w_before=one), lambda: norm(x.t()[:, :4], w_after=one),
                lambda: norm(x, gate=x[:3], w_after=one, w_before=one), lambda: norm(x, rows_per_gate=0, w_after=one),
                lambda: norm(x, gate=x, rows_per_gate=2, w_after=one, w_before=one),
                lambda: norm(x, w_after=one.half(), w_before=one)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dw.DwconvError):
        norm(x, w_before=one)  # no weight for the norm after the block
    conv.close()
    with pytest.raises(ValueError):
        conv(x, w)
