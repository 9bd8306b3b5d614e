"""The selective scan and the group norm on the GPU against the 64-bit
definitions, within the bounds of tests/scan_reference.py, through the binding's
classes."""
import pytest
import torch

import depthwise_convolution_amd as dw
import scan_reference as ref
import seq_reference
from gpu_helpers import DEV, say
from scan_cases import GROUP, SCAN, group_data, group_id, scan_data, scan_id
from depthwise_convolution_amd import seq
from seq_reference import DTYPES, U, starts

pytestmark = pytest.mark.gpu
NAMES = ("x", "dt", "a", "b", "c", "skip", "bias", "gate")
TAIL = 5  # tokens behind the last sequence


def up(t):
    return None if t is None else t.to(DEV)


def offsets_of(lens):
    return torch.tensor(starts(lens), dtype=torch.int32, device=DEV)


def wider(t, extra, value=float("nan")):
    """The same values as a slice of tokens with `extra` channels more, an odd number in front."""
    if t is None or not extra:
        return t
    n = t.shape[0]
    wide = torch.full((n, t[0].numel() + extra), value, dtype=t.dtype, device=t.device)
    view = wide[:, extra // 2:extra // 2 + t[0].numel()]
    view.copy_(t.reshape(n, -1))
    return view.unflatten(1, tuple(t.shape[1:])) if t.dim() > 2 else view


def tailed(t, extra):
    if t is None:
        return None
    return wider(torch.cat([t, torch.full((TAIL,) + tuple(t.shape[1:]), float("nan"), dtype=t.dtype)]).to(DEV), extra)


def holds(got, want, what):
    want, bound = want
    assert tuple(got.shape) == tuple(want.shape), what
    off = (got.double().cpu() - want).abs()
    worst = float((off / bound.clamp_min(1e-300)).max()) if off.numel() else 0.0
    print(f"{what}: worst {worst:.3f} of the bound", flush=True)
    assert not ref.outside(got, want, bound), what


def on_gpu(case, d):
    """Positional and named arguments, with tokens behind the last sequence and wider strides."""
    extra = case[9]
    pos = [tailed(d["x"], extra), tailed(d["dt"], extra), up(d["a"]), tailed(d["b"], extra), tailed(d["c"], extra)]
    return pos, dict(skip=up(d["skip"]), dt_bias=up(d["bias"]), gate=tailed(d["gate"], extra))


def plan_of(case):
    fmt, C, N, G, _, _, act, soft, _, _ = case
    return dw.SelectiveScan(C, N, G, fmt, softplus=soft, gate_act=act or "none")


@pytest.mark.parametrize("case", SCAN, ids=scan_id)
def test_scan_forward(case):
    fmt, C, N, G, lens, state, act, soft, _, extra = case
    say(f"[gpu] scan fwd {scan_id(case)}")
    d = scan_data(case, grad=False)
    T = sum(lens)
    pos, named = on_gpu(case, d)
    y = wider(torch.full((T + TAIL, C), 7.0, dtype=DTYPES[fmt], device=DEV), extra, 7.0)
    so = torch.full((len(lens), C, N), float("nan"), device=DEV)
    plan_of(case)(*pos, offsets=offsets_of(lens), state_in=up(d["state"]), state_out=so, y=y, **named)
    want = ref.scan_bounds(DTYPES[fmt], *(d[n] for n in NAMES), lens, d["state"], soft, act)
    holds(y[:T], want["y"], "y")
    holds(so, want["state"], "state")
    assert (y[T:] == 7.0).all(), "written behind the last sequence"
    if extra:
        base = y._base if y._base is not None else y
        assert int((base != 7.0).sum()) <= T * C, "written beside the channels"


@pytest.mark.parametrize("case", SCAN, ids=scan_id)
def test_scan_backward(case):
    fmt, C, N, G, lens, state, act, soft, _, extra = case
    say(f"[gpu] scan bwd {scan_id(case)}")
    d = scan_data(case, seed=3)
    T, dt = sum(lens), DTYPES[fmt]
    pos, named = on_gpu(case, d)
    full = lambda *s: wider(torch.full((T + TAIL,) + s, 7.0, dtype=dt, device=DEV), extra, 7.0)  # noqa: E731
    outs = dict(dx=full(C), ddt=full(C), db=full(G, N), dc=full(G, N))
    if act is not None:
        outs["dgate"] = full(C)
    g = plan_of(case).backward(*pos, tailed(d["dy"], extra), offsets=offsets_of(lens), state_in=up(d["state"]),
                               dstate_out=up(d["dstate"]), **outs, **named)
    got = dict(zip(("dx", "ddt", "da", "db", "dc", "dskip", "dbias", "dgate", "dstate"), g))
    want = ref.scan_bounds(dt, *(d[n] for n in NAMES), lens, d["state"], soft, act, d["dy"], d["dstate"])
    absent = {"dskip": d["skip"], "dbias": d["bias"], "dgate": d["gate"], "dstate": d["state"]}
    for k, v in got.items():
        if k in absent and absent[k] is None:
            assert v is None, k
            continue
        holds(v[:T] if k in outs else v, want[k], k)
        if k in outs:
            assert (v[T:] == 7.0).all(), f"{k}: written behind the last sequence"


def step_rows(case, rows, slots, seed=0):
    """One call of `rows` tokens, as sequences of their own: the rows of a slot in order."""
    fmt, C, N, G, _, _, act, soft, _, _ = case
    d = scan_data((fmt, C, N, G, [rows], False) + case[6:], seed=seed, grad=False)
    cache = torch.randn(max(slots) + 3, C, N, generator=torch.Generator().manual_seed(5)) * 0.5
    return d, cache


@pytest.mark.parametrize("case", SCAN[:12], ids=scan_id)
@pytest.mark.parametrize("slots", [None, [2, 0, 5, 9], [1, 4, 1, -1, 1, 4, 99, 0]], ids=["first", "given", "shared"])
def test_scan_step(case, slots):
    fmt, C, N, G, _, _, act, soft, _, extra = case
    say(f"[gpu] scan step {scan_id(case)} {slots}")
    rows = len(slots) if slots else 6
    at = slots or list(range(rows))
    d, cache = step_rows(case, rows, [s for s in at if s < 50])
    y = wider(torch.full((rows, C), 7.0, dtype=DTYPES[fmt], device=DEV), extra, 7.0)
    st = up(cache.clone())
    w = lambda t: wider(up(t), extra)  # noqa: E731
    plan_of(case).step(w(d["x"]), w(d["dt"]), up(d["a"]), w(d["b"]), w(d["c"]), st, skip=up(d["skip"]), dt_bias=up(d["bias"]),
                       gate=w(d["gate"]), slots=None if slots is None else torch.tensor(slots, dtype=torch.int32, device=DEV), y=y)
    for slot in range(cache.shape[0]):
        mine = [i for i, s in enumerate(at) if s == slot]
        if not mine:
            assert torch.equal(st[slot].cpu(), cache[slot])
            continue
        row = lambda t: None if t is None else t[mine]  # noqa: E731
        want = ref.scan_bounds(DTYPES[fmt], row(d["x"]), row(d["dt"]), d["a"], row(d["b"]), row(d["c"]), d["skip"], d["bias"],
                               row(d["gate"]), [len(mine)], cache[slot:slot + 1], soft, act)
        holds(y[mine], want["y"], f"y of slot {slot}")
        holds(st[slot:slot + 1], want["state"], f"state of slot {slot}")
    for i, s in enumerate(at):
        assert 0 <= s < cache.shape[0] or (y[i] == 7.0).all(), "a skipped row was written"


@pytest.mark.parametrize("fmt, C, N, G, rows, shared", [
    ("bf16", 2048, 16, 1, 203, False), ("bf16", 2048, 16, 1, 203, True), ("f16", 61, 11, 1, 4500, True),
    ("f32", 520, 100, 2, 97, True), ("f32", 300, 32, 3, 331, False)])
def test_scan_step_of_many_rows(fmt, C, N, G, rows, shared):
    """More rows than workgroups that walk them, slots that come again after many rows."""
    say(f"[gpu] scan step {fmt} {C} {N} {G} {rows} {shared}")
    case = (fmt, C, N, G, [], False, "silu", True, True, 0)
    entries = rows // 2 if shared else rows + 5
    g = torch.Generator().manual_seed(rows)
    at = torch.randint(-1, entries + 2, (rows,), generator=g) if shared else torch.randperm(entries, generator=g)[:rows]
    d, cache = step_rows(case, rows, [entries - 3])
    st, y = up(cache.clone()), torch.full((rows, C), 7.0, dtype=DTYPES[fmt], device=DEV)
    plan_of(case).step(up(d["x"]), up(d["dt"]), up(d["a"]), up(d["b"]), up(d["c"]), st, skip=up(d["skip"]),
                       dt_bias=up(d["bias"]), gate=up(d["gate"]), slots=up(at.to(torch.int32)), y=y)
    valid = (at >= 0) & (at < entries)
    order = torch.argsort(at, stable=True)
    order = order[valid[order]]  # a slot's rows together and in their order
    used, lens = torch.unique_consecutive(at[order], return_counts=True)
    row = lambda k: d[k][order]  # noqa: E731
    want = ref.scan_bounds(DTYPES[fmt], row("x"), row("dt"), d["a"], row("b"), row("c"), d["skip"], d["bias"], row("gate"),
                           lens.tolist(), cache[used], True, "silu")
    holds(y[up(order)], want["y"], "y")
    holds(st[up(used)], want["state"], "state")
    rest = torch.ones(entries, dtype=torch.bool)
    rest[used] = False
    assert torch.equal(st.cpu()[rest], cache[rest]) and (y[up(~valid)] == 7.0).all()


def test_scan_of_nothing():
    """No tokens, no sequences, only empty sequences."""
    C, N = 40, 16
    plan = dw.SelectiveScan(C, N, 1, "f32")
    e = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    a = -torch.ones(C, N, device=DEV)
    state = torch.randn(3, C, N, device=DEV)
    out = torch.full_like(state, float("nan"))
    y = plan(e(0, C), e(0, C), a, e(0, 1, N), e(0, 1, N), offsets=offsets_of([0, 0, 0]), state_in=state, state_out=out)
    assert y.shape == (0, C) and torch.equal(out, state)
    plan(e(0, C), e(0, C), a, e(0, 1, N), e(0, 1, N), offsets=offsets_of([0, 0, 0]), state_out=out)
    assert (out == 0).all()
    g = plan.backward(e(0, C), e(0, C), a, e(0, 1, N), e(0, 1, N), e(0, C), skip=e(C), dt_bias=e(C),
                      offsets=offsets_of([0, 0, 0]), state_in=state, dstate_out=state)
    assert torch.equal(g[8], state) and (g[2] == 0).all() and (g[5] == 0).all() and (g[6] == 0).all()
    y = plan(e(4, C), e(4, C), a, e(4, 1, N), e(4, 1, N), offsets=offsets_of([]), y=torch.full((4, C), 7.0, device=DEV))
    assert (y == 7.0).all()
    assert plan.step(e(0, C), e(0, C), a, e(0, 1, N), e(0, 1, N), state).shape == (0, C)


@pytest.mark.parametrize("T", [40, 900])
def test_wrong_offsets_stay_in_bounds(T):
    """Offsets that fall or run past the tokens are clamped, with whole sequences and with runs
    of them: what lies around the outputs and the workspace stays as it was."""
    C, N = 32, 16
    plan = dw.SelectiveScan(C, N, 1, "f32")
    g = torch.Generator().manual_seed(T)
    x, dt = up(torch.randn(T, C, generator=g)), up(torch.randn(T, C, generator=g))
    b, a = up(torch.randn(T, 1, N, generator=g)), -torch.ones(C, N, device=DEV)
    for bad in ([0, T + 500, 20], [-7, 10, 2 ** 30], [T - 5, 20, 10], [0, T, -1], [-2 ** 31, 2 ** 31 - 1, 3], [T + 9, T + 8, 0]):
        say(f"[gpu] scan offsets {bad}")
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        rows = [torch.full((T + 64, C), 5.0, device=DEV) for _ in range(3)]
        cols = [torch.full((T + 64, 1, N), 5.0, device=DEV) for _ in range(2)]
        states = [torch.full((4, C, N), 5.0, device=DEV) for _ in range(2)]
        y, dx, ddt = (v[32:32 + T] for v in rows)
        db, dc = (v[32:32 + T] for v in cols)
        so, ds = (v[1:3] for v in states)
        for back in (False, True):
            need = seq.dwconv_scan_workspace(plan.handle, 2, T, back)
            ws = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
            if back:
                plan.backward(x, dt, a, b, b, x, offsets=off, state_in=torch.zeros(2, C, N, device=DEV), dx=dx, ddt=ddt, db=db,
                              dc=dc, dstate_in=ds, workspace=ws[256:256 + need])
            else:
                plan(x, dt, a, b, b, offsets=off, state_out=so, y=y, workspace=ws[256:256 + need])
            torch.cuda.synchronize()
            assert (ws[:256] == 77).all() and (ws[256 + need:] == 77).all()
        for v in rows + cols:
            assert (v[:32] == 5.0).all() and (v[32 + T:] == 5.0).all()
        for v in states:
            assert (v[0] == 5.0).all() and (v[3] == 5.0).all()


def test_scan_repeats_its_bits_and_writes_states_in_place():
    case = ("bf16", 200, 16, 2, [300, 1, 90], True, "silu", True, True, 0)
    d = scan_data(case)
    pos, named = on_gpu(case, d)
    plan, off, dy = plan_of(case), offsets_of(case[4]), tailed(d["dy"], 0)
    T = sum(case[4])

    def both():
        st, ds = up(d["state"]), up(d["dstate"])
        y = plan(*pos, offsets=off, state_in=st, state_out=st, **named)
        g = plan.backward(*pos, dy, offsets=off, state_in=up(d["state"]), dstate_out=ds, dstate_in=ds, **named)
        return [y[:T], st, ds] + [v[:T] if v.shape[0] == T + TAIL else v for v in g]

    first = both()
    want = ref.scan_bounds(DTYPES["bf16"], *(d[n] for n in NAMES), case[4], d["state"], True, "silu", d["dy"], d["dstate"])
    holds(first[1], want["state"], "state in place")
    holds(first[2], want["dstate"], "dstate in place")
    for a, b in zip(first, both()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lens", [[40, 9], [700, 300], [64] * 13])
def test_scan_tokens_one_by_one(lens):
    """Steps over a cache give what the scan gives, within both bounds."""
    case = ("f32", 96, 16, 1, lens, True, "silu", True, True, 0)
    d = scan_data(case, grad=False)
    plan = plan_of(case)
    st = up(d["state"])
    y = torch.empty(sum(lens), 96, device=DEV)
    x, dt, b, c, z = (up(d[n]) for n in ("x", "dt", "b", "c", "gate"))
    a, skip, bias = up(d["a"]), up(d["skip"]), up(d["bias"])
    s = starts(lens)
    for t in range(max(lens)):
        rows = [i for i, n in enumerate(lens) if t < n]
        at = torch.tensor([s[i] + t for i in rows], device=DEV)
        y[at] = plan.step(x[at], dt[at], a, b[at], c[at], st, skip=skip, dt_bias=bias, gate=z[at],
                          slots=torch.tensor(rows, dtype=torch.int32, device=DEV))
    want = ref.scan_bounds(torch.float32, *(d[n] for n in NAMES), lens, d["state"])
    holds(y, want["y"], "y")
    holds(st, want["state"], "state")


@pytest.mark.parametrize("name", ["x", "dt", "gate", "b", "c", "state", "a"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("lens", [[40, 30], [300, 100]], ids=["whole", "runs"])
def test_scan_forward_is_causal_for_what_is_no_number(name, bad, lens):
    """A NaN or infinity reaches no token before its own, no other sequence and (but for
    b and c) no other channel; from its own token on its channel shows it."""
    case = ("bf16", 70, 16, 1, lens, True, "silu", True, True, 0)
    d = scan_data(case, seed=2, grad=False)
    plan, off, T = plan_of(case), offsets_of(lens), sum(lens)

    def run(d):
        pos, named = on_gpu(case, d)
        return plan(*pos, offsets=off, state_in=up(d["state"]), **named)[:T]

    clean = run(d)
    assert torch.isfinite(clean).all()
    for t in (0, 17, lens[0] - 1):
        e = {k: None if v is None else v.clone() for k, v in d.items()}
        ch = slice(69, 70)
        if name in ("b", "c"):
            e[name][t, 0, 3] = bad
            ch = slice(0, 70)
        elif name == "state":
            e["state"][0, 69, 3], t = bad, 0
        elif name == "a":
            e["a"][69, 3] = bad
        else:
            e[name][t, 69] = bad
        y = run(e)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[t:t + 1 if name in ("gate", "c") else lens[0], ch] = True
        if name == "a":
            hit[:, ch] = True
        assert torch.equal(y[~hit], clean[~hit]), (name, t)
        at = y[t, ch]
        assert not torch.isfinite(at).any() if name != "a" or bad != bad else True


def test_scan_rates_that_forget_or_keep_everything():
    """A rate of minus infinity keeps only the token itself; of zero, all of them."""
    C, N, T = 33, 16, 50
    d = scan_data(("f32", C, N, 1, [T], True, None, True, True, 0), grad=False)
    a = torch.zeros(C, N)
    a[:, ::2] = -float("inf")
    plan = dw.SelectiveScan(C, N, 1, "f32")
    st = torch.empty(1, C, N, device=DEV)
    y = plan(up(d["x"]), up(d["dt"]), up(a), up(d["b"]), up(d["c"]), state_in=up(d["state"]), state_out=st)
    width = ref.softplus(d["dt"].double())
    put = (width * d["x"].double())[:, :, None] * d["b"].double()
    h = d["state"].double() + put.cumsum(0)
    h[:, :, ::2] = put[:, :, ::2]
    want = (h * d["c"].double()).sum(-1)
    size = ((d["state"].double().abs() + put.abs().cumsum(0)) * d["c"].double().abs()).sum(-1)
    assert ((y.double().cpu() - want).abs() <= (T + 40) * U * size).all()
    assert ((st[0].double().cpu() - h[-1]).abs() <= (T + 40) * U * (d["state"][0].double().abs() + put.abs().sum(0))).all()


@pytest.mark.parametrize("soft", [True, False])
def test_scan_widths_far_from_zero(soft):
    """Widths from e^-80 to 80: one token of a zero state, h = d x b."""
    C, N = 4096, 1
    v = torch.linspace(-80, 80, C)
    plan = dw.SelectiveScan(C, N, 1, "f32", softplus=soft)
    one = torch.ones(1, C, device=DEV)
    st = torch.empty(1, C, N, device=DEV)
    b = torch.ones(1, 1, 1, device=DEV)
    plan(one, up(v[None]), torch.zeros(C, N, device=DEV), b, b, state_out=st)
    want = ref.softplus(v.double()) if soft else v.double()
    # exp2, its argument put right, the log's instruction and four roundings: 12 units
    assert ((st[0, :, 0].double().cpu() - want).abs() <= 12 * U * want.abs()).all()


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("case", GROUP, ids=group_id)
def test_group_forward(case):
    fmt, n, S, C, G, act, _, extra = case
    say(f"[gpu] group fwd {group_id(case)}")
    d = group_data(case)
    x = wider(up(d["x"]).view(n * S, C), extra).unflatten(0, (n, S))
    y = wider(torch.full((n * S, C), 7.0, dtype=DTYPES[fmt], device=DEV), extra + 2, 7.0).unflatten(0, (n, S))
    plan = dw.GroupNorm(C, G, fmt, act=act)
    plan(x, up(d["w"]), up(d["b"]), y=y)
    want = ref.group_bounds(DTYPES[fmt], d["x"], d["w"], d["b"], G, act, 1e-5)
    holds(y, want["y"], "y")
    assert int((y._base != 7.0).sum()) <= n * S * C, "written beside the channels"
    same = up(d["x"]).clone()
    assert plan(same, up(d["w"]), up(d["b"]), y=same) is same
    holds(same, want["y"], "in place")


@pytest.mark.parametrize("case", GROUP, ids=group_id)
def test_group_backward(case):
    fmt, n, S, C, G, act, params, extra = case
    say(f"[gpu] group bwd {group_id(case)}")
    d = group_data(case, seed=1)
    want = ref.group_bounds(DTYPES[fmt], d["x"], d["w"], d["b"], G, act, 1e-5, d["dy"])
    assert act != "relu" or want["border"] > 1, "a value of z within its error of the corner"
    wide = lambda t, e: wider(up(t).view(n * S, C), e).unflatten(0, (n, S))  # noqa: E731
    plan = dw.GroupNorm(C, G, fmt, act=act)
    dx, dw_, db = plan.backward(wide(d["x"], extra), wide(d["dy"], extra + 2 if extra else 0), up(d["w"]), up(d["b"]))
    holds(dx, want["dx"], "dx")
    assert (dw_ is None) == (d["w"] is None) and (db is None) == (d["b"] is None)
    if params:
        holds(dw_, want["dw"], "dw")
        holds(db, want["db"], "db")
    same = up(d["dy"]).clone()
    again = plan.backward(up(d["x"]), same, up(d["w"]), up(d["b"]), dx=same)
    assert again[0] is same
    holds(same, want["dx"], "in place")


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("size, eps", [(1e15, 1e-5), (1e-15, 0.0)])
@pytest.mark.parametrize("pixels", [60, 9000])
def test_group_of_far_sizes(act, size, eps, pixels):
    """Deviations whose squares are near fp32's ends."""
    d = group_data(("f32", 1, pixels, 48, 6, act, True, 0))
    x = d["x"] * size
    want = ref.group_bounds(torch.float32, x, d["w"], d["b"], 6, act, eps, d["dy"])
    plan = dw.GroupNorm(48, 6, "f32", act=act, eps=eps)
    holds(plan(up(x), up(d["w"]), up(d["b"])), want["y"], "y")
    for name, v in zip(("dx", "dw", "db"), plan.backward(up(x), up(d["dy"]), up(d["w"]), up(d["b"]))):
        holds(v, want[name], name)


@pytest.mark.parametrize("case", [c for c in GROUP if c[1] * c[2] * c[3] < 3e6], ids=group_id)
def test_group_workspaces_hold_what_a_call_keeps(case):
    fmt, n, S, C, G, act, _, _ = case
    d = group_data(case)
    x, dy, w, b = (up(d[k]) for k in ("x", "dy", "w", "b"))
    plan = dw.GroupNorm(C, G, fmt, act=act)
    for back in (False, True):
        need = seq.dwconv_group_workspace(plan.handle, n, S, back)
        ws = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
        if back:
            plan.backward(x, dy, w, b, workspace=ws[256:256 + need])
        else:
            plan(x, w, b, workspace=ws[256:256 + need])
        torch.cuda.synchronize()
        assert (ws[:256] == 77).all() and (ws[256 + need:] == 77).all()


def test_group_of_nothing():
    plan = dw.GroupNorm(8, 2, "f32")
    w = torch.ones(8, device=DEV)
    for shape in ((0, 5, 8), (3, 0, 8), (2, 0, 4, 8)):
        x = torch.zeros(shape, device=DEV)
        assert plan(x, w, w).shape == shape
        dx, dw_, db = plan.backward(x, x, w, w)
        assert dx.shape == shape and (dw_ == 0).all() and (db == 0).all()


def test_group_of_equal_values_and_of_none():
    """No variance: u is zero and y act(b); a NaN stays in its image and group."""
    plan = dw.GroupNorm(16, 4, "f32", act="none")
    x = torch.full((2, 40, 16), 3.0, device=DEV)
    b = torch.arange(16.0, device=DEV)
    assert torch.equal(plan(x, None, b), b.expand(2, 40, 16))
    x = torch.randn(2, 4000, 16, generator=torch.Generator().manual_seed(1)).to(DEV)
    clean = plan(x)
    x[1, 77, 5] = float("nan")
    y = plan(x)
    bad = y.isnan()
    assert bad[1, :, 4:8].all() and int(bad.sum()) == 4000 * 4 and torch.equal(y[~bad], clean[~bad])


def test_group_of_images_in_four_dimensions():
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(2, 5, 7, 24, generator=g)
    x = wide[..., 4:20]
    want = ref.group_bounds(torch.float32, x.reshape(2, 35, 16), None, None, 4, "silu", 1e-5)
    y = dw.GroupNorm(16, 4, "f32")(up(wide)[..., 4:20])
    assert y.shape == (2, 5, 7, 16)
    holds(y.view(2, 35, 16), want["y"], "y")


# ---------------------------------------------------------------------------
# as they are used: runs of operators, graphs, streams
# ---------------------------------------------------------------------------
def test_mixer_forward_and_gradients():
    """The short convolution, the scan behind it and the gated norm, and the gradients
    back through all three, against autograd of the definitions.  Each operator's output
    is rounded to fp32 (u) and met by sums of K + 1, then N + T tokens' and C terms;
    2-norms: 64 sqrt(T N) u."""
    C, K, N, lens = 48, 4, 16, [70, 1, 45]
    T = sum(lens)
    d = scan_data(("f32", C, N, 1, lens, True, "silu", True, True, 0), seed=9)
    g = torch.Generator().manual_seed(4)
    x, w, cb = torch.randn(T, C, generator=g), torch.randn(K, C, generator=g) * 0.5, torch.randn(C, generator=g) * 0.1
    nw = torch.rand(C, generator=g) + 0.5
    conv, scan = dw.CausalDepthwiseConv1d(C, K, "f32"), dw.SelectiveScan(C, N, 1, "f32")
    norm = dw.BlockNorm(C, "f32", after="rms", before="none", gate_act="none")
    off = offsets_of(lens)
    mixed = conv(up(x), up(w), up(cb), offsets=off)
    args = (mixed, up(d["dt"]), up(d["a"]), up(d["b"]), up(d["c"]))
    named = dict(skip=up(d["skip"]), dt_bias=up(d["bias"]), gate=up(d["gate"]), offsets=off)
    y = scan(*args, **named)
    out, _ = norm(y, w_after=up(nw))
    dy, _, _, _, dnw, _, _, _ = norm.backward(y, dh=up(d["dy"]), w_after=up(nw))
    dmixed, ddt, da, db, dc, dskip, dbias, dgate, _ = scan.backward(*args, dy, **named)
    dx, dwt, dcb, _ = conv.backward(up(x), up(w), dmixed, up(cb), offsets=off)
    ls = seq_reference.leaves(x, w, cb, d["dt"], d["a"], d["b"], d["c"], d["skip"], d["bias"], d["gate"], nw)
    m = seq_reference.conv(ls[0], ls[1], ls[2], lens, None, "silu")[0]
    s = ref.scan(m, *ls[3:10], lens, None)[0]
    want = seq_reference.normed(s, "rms", ls[10], None, 1e-6)
    tol = 64 * (T * N) ** 0.5 * U
    assert seq_reference.rel(out.cpu(), want.detach()) <= tol
    grads = torch.autograd.grad(want, ls, d["dy"].double())
    for n, a, b in zip("x w cb dt a b c skip bias gate nw".split(), (dx, dwt, dcb, ddt, da, db, dc, dskip, dbias, dgate, dnw),
                       grads):
        assert seq_reference.rel(a.cpu(), b) <= tol, n


def test_image_block():
    """A depthwise convolution and the group norm with its activation behind it, and the
    gradients of both."""
    N, H, W, C = 2, 12, 10, 32
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(N, H, W, C, generator=g), torch.randn(3, 3, C, generator=g) / 3
    gw, gb, dz = torch.rand(C, generator=g) + 0.5, torch.randn(C, generator=g) * 0.2, torch.randn(N, H, W, C, generator=g)
    conv = dw.DepthwiseConv2d(N=N, H=H, W=W, C=C, FH=3, FW=3, stride=1, dilation=1, pad=1, dtype="f32")
    group = dw.GroupNorm(C, 8, "f32", act="silu")
    y = conv(up(x), up(w), torch.zeros(C, device=DEV))
    z = group(y, up(gw), up(gb))
    dy, dgw, dgb = group.backward(y, up(dz), up(gw), up(gb))
    dx, dwt = conv.backward_data(dy, up(w)), conv.backward_filter(up(x), dy)
    ls = seq_reference.leaves(x, w, gw, gb)
    cy = torch.nn.functional.conv2d(ls[0].permute(0, 3, 1, 2), ls[1].permute(2, 0, 1)[:, None], padding=1, groups=C)
    cz = ref.group(cy.permute(0, 2, 3, 1).reshape(N, H * W, C), ls[2], ls[3], 8, "silu", 1e-5).view(N, H, W, C)
    tol = 64 * (H * W) ** 0.5 * U
    assert seq_reference.rel(z.cpu(), cz.detach()) <= tol
    for a, b in zip((dx, dwt, dgw, dgb), torch.autograd.grad(cz, ls, dz.double())):
        assert seq_reference.rel(a.cpu(), b) <= tol


def calls():
    """name: (fn(stream), outputs) over fixed tensors."""
    case = ("bf16", 320, 16, 1, [700, 30], True, "silu", True, True, 0)
    d = scan_data(case)
    pos, named = on_gpu(case, d)
    plan, off, dy = plan_of(case), offsets_of(case[4]), tailed(d["dy"], 0)
    st, dst = up(d["state"]), up(d["dstate"])
    cache = torch.randn(800, 320, 16, device=DEV) * 0.1
    x = torch.randn(3, 400, 96, device=DEV)
    big = torch.randn(2, 9000, 48, device=DEV)
    w, b = torch.rand(96, device=DEV), torch.rand(96, device=DEV)
    norm, wide, plain = dw.GroupNorm(96, 32, "f32"), dw.GroupNorm(48, 6, "f32"), dw.GroupNorm(48, 6, "f32", act="none")
    T = sum(case[4])
    out = torch.zeros(T + TAIL, 320, dtype=torch.bfloat16, device=DEV)
    so = torch.zeros_like(st)

    def fwd(s):
        plan(*pos, offsets=off, state_in=st, state_out=so, y=out, stream=s, **named)
        return [out[:T], so]

    return {
        "scan forward": fwd,
        "scan step": lambda s: [plan.step(*(t[:T] if t.shape[0] > 320 else t for t in pos), cache, skip=named["skip"],
                                          dt_bias=named["dt_bias"], gate=named["gate"][:T], stream=s)],
        "scan backward": lambda s: [v[:T] if v.shape[0] == T + TAIL else v for v in plan.backward(
            *pos, dy, offsets=off, state_in=st, dstate_out=dst, stream=s, **named)],
        "group forward": lambda s: [norm(x, w, b, stream=s), wide(big, stream=s)],
        "group backward": lambda s: list(norm.backward(x, x, w, b, stream=s)) + [wide.backward(big, big, stream=s)[0]]
        + list(plain.backward(big, big, w[:48], b[:48], stream=s)),
    }


@pytest.mark.parametrize("name", ["scan forward", "scan backward", "group forward", "group backward"])
def test_replayed_graphs(name):
    """Two graphs of the same call, replayed in turn with eager calls between, give its bits."""
    say(f"[gpu] graph {name}")
    fn = calls()[name]
    want = [t.clone() for t in fn(None)]
    side = torch.cuda.Stream()
    graphs = []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn(None)
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = fn(None)
            graphs.append((g, out))
    torch.cuda.synchronize()
    for turn in range(3):
        for g, out in graphs:
            for t in out:
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (name, turn)
        assert all(torch.equal(a, b) for a, b in zip(fn(None), want))


def test_replayed_steps():
    """A captured step moves its cache with every replay as eager calls do theirs."""
    C, N, rows = 512, 16, 150
    d, cache = step_rows(("bf16", C, N, 1, [], False, "silu", True, True, 0), rows, [rows])
    args = [up(d[k]) for k in ("x", "dt", "a", "b", "c")]
    named = dict(skip=up(d["skip"]), dt_bias=up(d["bias"]), gate=up(d["gate"]),
                 slots=up((torch.arange(rows) * 7 % 100).to(torch.int32)))
    plan = dw.SelectiveScan(C, N, 1, "bf16")
    eager, st = up(cache.clone()), up(cache.clone())
    y = torch.empty(rows, C, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        plan.step(*args, st, y=y, **named)
    torch.cuda.synchronize()
    assert torch.equal(st, eager), "capturing ran it"
    for turn in range(3):
        want = plan.step(*args, eager, **named)
        torch.cuda.synchronize()
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(st, eager), turn


@pytest.mark.parametrize("name", ["scan forward", "scan step", "scan backward", "group forward", "group backward"])
def test_given_streams(name):
    """On a stream of its own, on its raw handle, and two calls at once on two streams."""
    say(f"[gpu] streams {name}")
    torch.manual_seed(11)
    fn = calls()[name]
    if name == "scan step":  # the cache moves with every call: only that it runs there
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        y = fn(s)[0]
        torch.cuda.current_stream().wait_stream(s)
        assert torch.isfinite(y).all()
        return
    want = [t.clone() for t in fn(None)]
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    raw = fn(one.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(raw, want))
    a, b = fn(one), fn(two)
    torch.cuda.synchronize()
    for out in (a, b):
        assert all(torch.equal(p, q) for p, q in zip(out, want))
