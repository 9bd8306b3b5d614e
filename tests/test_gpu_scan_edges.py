"""The selective scan and the group norm on the GPU where tests/test_gpu_scan.py does not
reach: states that grow, long runs, every number of lanes a channel, wide slices, streams."""
import pytest
import torch

import depthwise_convolution_amd as dw
import scan_reference as ref
import test_gpu_scan as base
from gpu_helpers import DEV, say
from scan_cases import SCAN, group_data, group_id, scan_data, scan_id
from scan_long import LONG, long_bounds, long_data, long_id
from depthwise_convolution_amd import seq
from seq_reference import DTYPES, U, leaves, starts

pytestmark = pytest.mark.gpu


def up(t):
    return None if t is None else t.to(DEV)


# ---------------------------------------------------------------------------
# states that grow
# ---------------------------------------------------------------------------
LEAST = 2.0 ** -126  # fp32's least normal number, below which values may be flushed


def growing(T, C, N, x_at, dy_at, small, falling):
    """Positive values throughout, so that each result is the size of its terms.  Exponents d a
    of 0.5 to 2 a token, 64 to 128 a run of 64 tokens (e^88.7 is fp32's end): rates above zero,
    or (``falling``) below it with widths below it.  x and dy are zero but at their tokens."""
    g = torch.Generator().manual_seed(T + C)
    r = lambda *s: 0.5 + torch.rand(*s, generator=g)  # noqa: E731
    only = lambda at: r(T, C) * torch.isin(torch.arange(T), torch.tensor(at, dtype=torch.long))[:, None]  # noqa: E731
    a, dt = 1 + r(C, N) * 0.6, 0.8 + 0.2 * r(T, C)
    d = dict(x=only(x_at), dt=dt, a=a, b=r(T, 1, N), c=r(T, 1, N), dy=only(dy_at), state=None, dstate=None)
    if falling:
        d.update(a=-a, dt=-dt, x=-d["x"])
    if small:
        d["state"], d["dstate"] = r(1, C, N) * small[0], r(1, C, N) * small[1]
    return d


def near(got, want, tol, what):
    want = want.detach()
    off = (got.double().cpu() - want).abs()
    worst = float((off / (tol * want.abs() + 16 * LEAST)).max())
    print(f"{what}: worst {worst:.3f} of the bound", flush=True)
    assert worst <= 1, what


@pytest.mark.parametrize("falling", [False, True], ids=["rates", "widths"])
@pytest.mark.parametrize("T, C, N, x_at, dy_at, small", [
    (2048, 64, 16, [2040, 2047], [1, 5], None),           # zero states and gradients past many runs
    (300, 33, 5, [297, 299], [0, 3], None),
    (400, 40, 30, [395], [6], None),
    (330, 20, 100, [326, 328], [0, 2], None),
    (68, 40, 16, [], [], (2.0 ** -120, 2.0 ** -120)),     # small ones that a run takes past e^100
])
def test_scan_of_states_that_grow(T, C, N, x_at, dy_at, small, falling):
    """A run's factor beyond fp32's range: zero states stay zero, small ones arrive.

    Every value is a sum of positive products, so its relative error is that of its largest
    factor: exponents X = sum |d a| along the way, each off by 21 u of itself (a run's widths
    are added 16 to a lane, then over four lanes: 18; rates times log2 e, products and halves:
    3), three roundings a token (exponential, state and input), sums over N states, C channels
    and T tokens: (21 X + 4 T + N + C + 40) u, with X at most 2.5 for each token between the
    first and the last that is not zero."""
    say(f"[gpu] scan growth {T} {C} {N} {falling}")
    d = growing(T, C, N, x_at, dy_at, small, falling)
    plan = dw.SelectiveScan(C, N, 1, "f32", softplus=False, gate_act="none")
    pos = [up(d[k]) for k in ("x", "dt", "a", "b", "c")]
    so = torch.empty(1, C, N, device=DEV)
    y = plan(*pos, state_in=up(d["state"]), state_out=so)
    zero = torch.zeros(1, C, N)
    g = plan.backward(*pos, up(d["dy"]), state_in=up(zero if d["state"] is None else d["state"]), dstate_out=up(d["dstate"]))
    state = zero if d["state"] is None else d["state"]
    ls = leaves(d["x"], d["dt"], d["a"], d["b"], d["c"], state)
    wy, ws = ref.scan(*ls[:5], None, None, None, [T], ls[5], soft=False, act="none")
    outs, gives = [wy], [d["dy"].double()]
    if d["dstate"] is not None:
        outs, gives = outs + [ws], gives + [d["dstate"].double()]
    grads = torch.autograd.grad(outs, ls, gives)
    tol = (21 * 2.5 * (T if small else 10) + 4 * T + N + C + 40) * U
    near(y, wy, tol, "y")
    near(so, ws, tol, "state")
    for name, got, want in zip(("dx", "ddt", "da", "db", "dc", "dstate"), g[:5] + g[8:], grads):
        near(got, want, tol, name)


# ---------------------------------------------------------------------------
# every number of lanes a channel, type and gate, whole sequences and runs; long runs
# ---------------------------------------------------------------------------
# as SCAN in tests/scan_cases.py
LANES = [
    ("f32", 70, 24, 1, [33, 40, 2], True, "silu", True, True, 0),          # 8 lanes a channel, whole
    ("f16", 64, 32, 2, [40, 1, 0, 33], True, "silu", True, True, 0),
    ("bf16", 61, 19, 1, [50, 17], False, "sigmoid", True, True, 3),
    ("f32", 33, 17, 1, [50, 30], True, None, True, True, 0),
    ("f16", 40, 30, 1, [64, 3], True, None, False, True, 1),
    ("f32", 33, 20, 1, [300], True, "silu", True, True, 0),                # and in runs
    ("f16", 50, 17, 1, [400, 5], True, "sigmoid", True, True, 0),
    ("bf16", 96, 32, 3, [300, 10], True, "silu", True, True, 5),
    ("bf16", 40, 25, 1, [200], True, None, True, False, 0),
    ("bf16", 512, 24, 1, [3, 5, 0, 1] * 500, True, "silu", True, True, 0),  # more sequences than walkers of the gradients
    ("f32", 24, 64, 2, [40, 33], True, "silu", True, True, 0),             # 16 lanes
    ("bf16", 17, 33, 1, [30, 50], True, "silu", True, True, 0),
    ("f16", 40, 48, 1, [50, 40], True, "sigmoid", True, True, 0),
    ("f32", 20, 40, 1, [200, 9], True, "silu", True, True, 0),
    ("bf16", 36, 50, 2, [250], True, "silu", True, True, 2),
    ("f16", 12, 70, 1, [40, 9], True, "silu", True, True, 0),              # 32 lanes
    ("f32", 9, 128, 1, [30, 41], True, "silu", True, True, 0),
    ("bf16", 20, 66, 2, [33, 1], False, None, True, True, 0),
    ("f16", 10, 65, 1, [200, 70], True, "silu", True, True, 1),
    ("bf16", 11, 127, 1, [300], True, "sigmoid", True, True, 0),
]


@pytest.mark.parametrize("case", LANES, ids=scan_id)
def test_scan_forward_of_any_lanes(case):
    base.test_scan_forward(case)


@pytest.mark.parametrize("case", LANES, ids=scan_id)
def test_scan_backward_of_any_lanes(case):
    base.test_scan_backward(case)


@pytest.mark.parametrize("case", LONG, ids=long_id)
def test_scan_in_long_runs(case):
    """Runs of 128 to 1024 tokens, half of the states slow enough to pass from one to the next.
    Inputs of one sign, whose sums are not smaller than their terms."""
    fmt, C, N, G, lens, act, run = case
    say(f"[gpu] scan long {long_id(case)}")
    d = long_data(case)
    T, dt = sum(lens), DTYPES[fmt]
    plan, off = dw.SelectiveScan(C, N, G, fmt, gate_act=act), base.offsets_of(lens)
    pos = [up(d[k]) for k in ("x", "dt", "a", "b", "c")]
    named = dict(skip=up(d["skip"]), dt_bias=up(d["bias"]), gate=up(d["gate"]), offsets=off, state_in=up(d["state"]))
    so = torch.empty(len(lens), C, N, device=DEV)
    y = plan(*pos, state_out=so, **named)
    got = dict(zip(("dx", "ddt", "da", "db", "dc", "dskip", "dbias", "dgate", "dstate"),
                   plan.backward(*pos, up(d["dy"]), dstate_out=up(d["dstate"]), **named)), y=y, state=so)
    torch.cuda.synchronize()
    # a sum over tokens: a run's, then four chains of up to 2048 walkers' in all
    wants = []
    for i, (s, n) in enumerate(zip(starts(lens), lens)):
        cut = lambda t: t[s:s + n]  # noqa: E731
        wants.append(long_bounds(dt, cut(d["x"]), cut(d["dt"]), d["a"], cut(d["b"]), cut(d["c"]), d["skip"], d["bias"],
                                 cut(d["gate"]), d["state"][i], True, act, cut(d["dy"]), d["dstate"][i], run + 512 + 8))
    for k, v in got.items():
        whole = k in ("da", "dskip", "dbias")
        want = tuple(sum(w[k][j] for w in wants) if whole else torch.cat([w[k][j] for w in wants]) for j in (0, 1))
        base.holds(v, want, k)


# ---------------------------------------------------------------------------
# group norm: wide slices, far means
# ---------------------------------------------------------------------------
# as GROUP in tests/scan_cases.py: groups in no number that divides well, so that a slice is all
# channels and its lanes' values, columns and statistics take 64 to 128 KB of LDS
WIDE = [
    ("bf16", 1, 9, 8192, 1, "silu", True, 0),
    ("bf16", 2, 9, 4099, 4099, "none", True, 0),
    ("f16", 1, 32, 4093, 4093, "silu", True, 0),
    ("f16", 1, 9, 6002, 3001, "relu", True, 0),
    ("bf16", 2, 16, 8191, 8191, "silu", True, 3),
]


@pytest.mark.parametrize("case", WIDE, ids=group_id)
def test_group_forward_of_wide_slices(case):
    fmt, n, S, C, G, act, _, _ = case
    assert seq.dwconv_group_workspace(dw.GroupNorm(C, G, fmt, act=act).handle, n, S, False) == 0, "not in registers"
    base.test_group_forward(case)


@pytest.mark.parametrize("case", WIDE, ids=group_id)
def test_group_backward_of_wide_slices(case):
    base.test_group_backward(case)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("fmt, mean", [("f32", 1000.0), ("f32", 30.0), ("f16", 30.0), ("bf16", 10.0)])
@pytest.mark.parametrize("pixels", [60, 9000])
def test_group_of_means_far_from_zero(fmt, mean, pixels, act):
    """Means of up to 1000 deviations: x r - mean r loses what the mean itself does, and the
    bounds have it."""
    say(f"[gpu] group far mean {fmt} {mean} {pixels} {act}")
    d = group_data((fmt, 2, pixels, 48, 6, act, True, 0), seed=4)
    x = (torch.randn(2, pixels, 48, generator=torch.Generator().manual_seed(6)) + mean).to(DTYPES[fmt])
    want = ref.group_bounds(DTYPES[fmt], x, d["w"], d["b"], 6, act, 1e-5, d["dy"])
    plan = dw.GroupNorm(48, 6, fmt, act=act)
    base.holds(plan(up(x), up(d["w"]), up(d["b"])), want["y"], "y")
    for name, v in zip(("dx", "dw", "db"), plan.backward(up(x), up(d["dy"]), up(d["w"]), up(d["b"]))):
        base.holds(v, want[name], name)


@pytest.mark.parametrize("act", ["none", "silu", "relu"])
@pytest.mark.parametrize("fmt, C", [("f32", 64), ("bf16", 64), ("f16", 40), ("f32", 3), ("bf16", 5), ("f16", 1)])
def test_group_of_one_value(fmt, C, act):
    """A group that is one value has u = 0 whatever the value is: y = act(b), and nothing
    depends on x or w.  (Channels in vectors, and too few for one.)"""
    say(f"[gpu] group of one {fmt} {C} {act}")
    g, dt = torch.Generator().manual_seed(C), DTYPES[fmt]
    x, dy = up((torch.randn(1, 1, C, generator=g) * 5 + 20).to(dt)), up(torch.randn(1, 1, C, generator=g).to(dt))
    w, b = up(0.5 + torch.rand(C, generator=g)), up(torch.randn(C, generator=g))
    plan = dw.GroupNorm(C, C, fmt, act=act)
    zero = torch.zeros_like(x)
    assert torch.equal(plan(x, w, b), plan(zero, None, b))
    if act != "silu":
        assert torch.equal(plan(x, w, b)[0, 0], (b if act == "none" else b.clamp_min(0)).to(dt))
    dx, dw_, db = plan.backward(x, dy, w, b)
    assert (dx == 0).all() and (dw_ == 0).all()
    assert torch.equal(db, plan.backward(zero, dy, w, b)[2])
    if act == "none":
        assert torch.equal(db, dy[0, 0].float())


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("pixels, C, G", [(49, 48, 6), (9000, 48, 6), (3000, 61, 61), (500, 7, 1), (20000, 256, 2)])
def test_group_of_equal_values(pixels, C, G, act):
    """Images without variance whose sums are exact (8 bits of bf16 times up to 2^15 values of
    a workgroup): u = 0 to the last bit, in registers and in passes, whatever their value is."""
    say(f"[gpu] group of equals {pixels} {C} {G} {act}")
    g = torch.Generator().manual_seed(pixels)
    value = (torch.randn(2, 1, G, generator=g) * 5 + 20).to(torch.bfloat16).repeat_interleave(C // G, 2)
    x, dy = up(value.expand(2, pixels, C).contiguous()), up(torch.randn(2, pixels, C, generator=g).to(torch.bfloat16))
    w, b = up(0.5 + torch.rand(C, generator=g)), up(torch.randn(C, generator=g))
    plan = dw.GroupNorm(C, G, "bf16", act=act)
    y, dw_ = plan(x, w, b), plan.backward(x, dy, w, b)[1]
    assert torch.equal(y, plan(torch.zeros_like(x), None, b))
    assert act != "none" or torch.equal(y, b.bfloat16().expand_as(y))
    assert (dw_ == 0).all()


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("pixels", [60, 9000])
def test_group_of_what_is_no_number_or_too_large(pixels, act):
    """A NaN or infinity makes NaN of its image's group and of nothing else; deviations whose
    squares leave fp32 have u = 0."""
    plan, g = dw.GroupNorm(48, 6, "f32", act=act), torch.Generator().manual_seed(pixels)
    x, dy = up(torch.randn(2, pixels, 48, generator=g)), up(torch.randn(2, pixels, 48, generator=g))
    w, b = up(0.5 + torch.rand(48, generator=g)), up(torch.randn(48, generator=g))
    clean = plan(x, w, b), plan.backward(x, dy, w, b)[0]
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[1, :, :8] = True
    for bad in (float("nan"), float("inf"), -float("inf")):
        e = x.clone()
        e[1, 7, 5] = bad
        for got, was in zip((plan(e, w, b), plan.backward(e, dy, w, b)[0]), clean):
            assert got[hit].isnan().all() and torch.equal(got[~hit], was[~hit]), bad
    x[1] *= 1e20
    y, (dx, dw_, db) = plan(x, w, b), plan.backward(x, dy, w, b)
    zero = plan(torch.zeros_like(x), None, b)
    assert torch.equal(y[1], zero[1]) and (dx[1] == 0).all() and torch.equal(y[0], clean[0][0])
    assert torch.isfinite(dw_).all() and torch.isfinite(db).all()
    x[1] = 1e38  # 60 x 8 of them add up to more than fp32 holds
    y, dx = plan(x, w, b), plan.backward(x, dy, w, b)[0]
    assert y[1].isnan().all() and dx[1].isnan().all() and torch.equal(y[0], clean[0][0]) and torch.equal(dx[0], clean[1][0])


# ---------------------------------------------------------------------------
# workspaces and streams
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("case", SCAN + LANES, ids=scan_id)
def test_scan_workspaces_hold_what_a_call_keeps(case):
    """What lies around a workspace of just its size stays as it was."""
    fmt, C, N, G, lens, state, act, soft, _, _ = case
    say(f"[gpu] scan workspace {scan_id(case)}")
    d = scan_data(case)
    plan, off = base.plan_of(case), base.offsets_of(lens)
    pos = [up(d[k]) for k in ("x", "dt", "a", "b", "c")]
    named = dict(skip=up(d["skip"]), dt_bias=up(d["bias"]), gate=up(d["gate"]), offsets=off, state_in=up(d["state"]))
    for back in (False, True):
        need = seq.dwconv_scan_workspace(plan.handle, len(lens), sum(lens), back)
        ws = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
        if back:
            plan.backward(*pos, up(d["dy"]), dstate_out=up(d["dstate"]), workspace=ws[256:256 + need], **named)
        else:
            plan(*pos, state_out=torch.empty(len(lens), C, N, device=DEV), workspace=ws[256:256 + need], **named)
        torch.cuda.synchronize()
        assert (ws[:256] == 77).all() and (ws[256 + need:] == 77).all()


def stream_calls():
    """name: (outputs that no call has written, call(stream, outputs)); the step's cache holds
    its states."""
    case = ("bf16", 320, 16, 1, [700, 30], True, "silu", True, True, 0)
    d = {k: up(v) for k, v in scan_data(case).items()}
    plan, off, T, bf = base.plan_of(case), base.offsets_of(case[4]), 730, torch.bfloat16
    pos = [d[k] for k in ("x", "dt", "a", "b", "c")]
    named = dict(skip=d["skip"], dt_bias=d["bias"], gate=d["gate"])
    cache = torch.randn(800, 320, 16, device=DEV) * 0.1
    x, big = torch.randn(3, 400, 96, device=DEV), torch.randn(2, 9000, 48, device=DEV)
    w, b = torch.rand(96, device=DEV), torch.rand(96, device=DEV)
    plans = [(dw.GroupNorm(96, 32, "f32"), x, 96), (dw.GroupNorm(48, 6, "f32"), big, 48),
             (dw.GroupNorm(48, 6, "f32", act="none"), big, 48)]
    none = lambda *s, dtype=torch.float32: torch.full(s, float("nan"), dtype=dtype, device=DEV)  # noqa: E731
    rows, cols = lambda: none(T, 320, dtype=bf), lambda: none(T, 1, 16, dtype=bf)  # noqa: E731
    grads = "dx ddt da db dc dskip ddt_bias dgate dstate_in".split()

    def group_fwd(s, o):
        for (p, v, C), y in zip(plans, o):
            p(v, w[:C], b[:C], y=y, stream=s)

    def group_bwd(s, o):
        for i, (p, v, C) in enumerate(plans):
            p.backward(v, v, w[:C], b[:C], dx=o[3 * i], dw=o[3 * i + 1], db=o[3 * i + 2], stream=s)

    return {
        "scan forward": (lambda: [rows(), none(2, 320, 16)], lambda s, o: plan(
            *pos, offsets=off, state_in=d["state"], y=o[0], state_out=o[1], stream=s, **named)),
        "scan step": (lambda: [rows(), cache.clone()], lambda s, o: plan.step(*pos, o[1], y=o[0], stream=s, **named)),
        "scan backward": (lambda: [rows(), rows(), none(320, 16), cols(), cols(), none(320), none(320), rows(), none(2, 320, 16)],
                          lambda s, o: plan.backward(*pos, d["dy"], offsets=off, state_in=d["state"], dstate_out=d["dstate"],
                                                     stream=s, **dict(zip(grads, o)), **named)),
        "group forward": (lambda: [torch.full_like(v, float("nan")) for _, v, _ in plans], group_fwd),
        "group backward": (lambda: [t for _, v, C in plans for t in (torch.full_like(v, float("nan")), none(C), none(C))],
                           group_bwd),
    }


@pytest.mark.parametrize("name", ["scan forward", "scan step", "scan backward", "group forward", "group backward"])
def test_outputs_of_calls_on_given_streams(name):
    """Every call writes outputs of its own, of which none holds the values before: on a raw
    handle, on two streams at once, and on a stream that is busy, of which the current one sees
    nothing yet."""
    say(f"[gpu] given streams {name}")
    torch.manual_seed(3)
    make, call = stream_calls()[name]
    want, one, two = make(), torch.cuda.Stream(), torch.cuda.Stream()
    call(None, want)
    equal = lambda o: all(torch.equal(p, q) for p, q in zip(o, want))  # noqa: E731
    sets = [make() for _ in range(3)]
    untouched = make()
    m = torch.ones(8192, 8192, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in want) and not any(equal(o) for o in sets)
    call(one.cuda_stream, sets[0])
    torch.cuda.synchronize()
    assert equal(sets[0])
    call(one, sets[1])
    call(two, sets[2])
    torch.cuda.synchronize()
    assert equal(sets[1]) and equal(sets[2])
    for _ in range(4):  # streams that share a hardware queue with the current one are no test of this
        given, out = torch.cuda.Stream(), make()
        busy, saw = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        with torch.cuda.stream(given):
            for _ in range(100):
                torch.mm(m, m)
            busy.record()
        call(given, out)
        seen = [t.clone() for t in out]
        saw.record()
        torch.cuda.synchronize()
        assert equal(out)
        early = saw.elapsed_time(busy)
        print(f"{name}: seen {early:.2f} ms before the given stream was free", flush=True)
        if early > 0:
            same = [bool((p.nan_to_num(7.0) == q.nan_to_num(7.0)).all()) for p, q in zip(seen, untouched)]
            assert all(same), "written by another stream than the given one"
            return
    pytest.skip("no stream ran beside the current one")
