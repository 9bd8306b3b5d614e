"""The sequence operators on the GPU where they are easily wrong: sums that
cancel, values that are not numbers, borders.  Bounds are derived in
tests/seq_cases.py and shown on planted mistakes in tests/test_seq_bounds.py."""
import pytest
import torch

import depthwise_convolution_amd as dw
import seq_reference as ref
from gpu_helpers import DEV, say
from seq_cases import CONV_GRADS, conv_grad_bounds, conv_grad_data, readback, readback_bound, readback_terms
from seq_reference import leaves, rel
import test_gpu_seq
from test_gpu_seq import delta_data, offsets_of, rand, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,Hk,Hv,Dk,Dv,lens", [
    ("bf16", 1, 2, 128, 48, [64, 70, 3]), ("f16", 1, 2, 128, 48, [64, 70, 3]), ("f32", 1, 2, 128, 48, [64, 70, 3]),
    ("bf16", 2, 2, 64, 33, [130]), ("f16", 1, 1, 64, 64, [1, 65]), ("bf16", 1, 1, 192, 40, [100]),
    ("f16", 1, 1, 192, 40, [100]), ("bf16", 1, 1, 256, 40, [100]), ("f16", 1, 1, 256, 32, [70]),
    ("bf16", 1, 3, 128, 70, [66, 64, 1] * 20), ("f16", 1, 3, 100, 70, [66, 64, 1] * 20),
], ids=str)
def test_delta_reads_back_what_it_stored(fmt, Hk, Hv, Dk, Dv, lens):
    """Outputs that are a small difference of large terms keep fp32 accuracy of
    the terms, whatever type o is rounded to."""
    say(f"[gpu] delta read-back {fmt} {Hk} {Hv} {Dk} {Dv} {lens[:4]}")
    q, k, v, g, beta, state = readback(fmt, Hk, Hv, Dk, Dv, lens)
    scale = Dk ** -0.5
    o = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, fmt)(*(up(t) for t in (q, k, v, g, beta)), offsets=offsets_of(lens),
                                               state_in=up(state))
    want, _, _ = ref.delta(*(t.double() for t in (q, k, v, g, beta)), lens, state.double(), scale, True, 1e-6)
    c = readback_terms(q, k, lens, state, v, scale, 1e-6)
    off, bound = float((o.double().cpu() - want).norm()), readback_bound(v.dtype, want, c, Dk)
    print(f"{fmt} Dk={Dk}: off {off / bound:.2f} of the bound", flush=True)
    assert off <= bound


# ---------------------------------------------------------------------------
# values that are not numbers
# ---------------------------------------------------------------------------
NAN, INF = float("nan"), float("inf")
SPOIL = [("v", NAN), ("v", INF), ("v", -INF), ("k", NAN), ("k", INF), ("q", NAN), ("beta", NAN), ("g", NAN),
         ("state", NAN), ("beta", INF)]


def of_head(name, h, group):
    """The value heads that head h of tensor `name` belongs to."""
    return list(range(h * group, (h + 1) * group)) if name in ("q", "k") else [h]


@pytest.mark.parametrize("name,bad", SPOIL, ids=lambda x: str(x))
@pytest.mark.parametrize("fmt,Hk,Hv,Dk,Dv,lens,chunk_first", [
    ("f32", 1, 2, 40, 70, [130, 70], 64), ("bf16", 1, 2, 128, 70, [130, 70], 64), ("f16", 2, 4, 64, 40, [130, 70], 64),
    ("bf16", 1, 3, 100, 70, [130, 70] * 16, 64), ("f16", 1, 1, 250, 33, [130, 70], 0), ("bf16", 1, 5, 72, 24, [90, 70], 64),
], ids=lambda x: str(x)[:12])
def test_delta_forward_is_causal_for_what_is_no_number(fmt, Hk, Hv, Dk, Dv, lens, chunk_first, name, bad):
    """A NaN or infinity at token t: the outputs of the tokens before it, of other
    sequences, other heads and (for v and the state) other columns keep their
    bits; its own and the later ones of its column are no numbers either."""
    say(f"[gpu] delta spoiled {fmt} {Hk} {Hv} {Dk} {Dv} {name} {bad}")
    data = [t for t in delta_data(fmt, Hk, Hv, Dk, Dv, lens, True, gates="plain", seed=7)]
    names = ["q", "k", "v", "g", "beta", "state"]
    rule, off, group = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, fmt), offsets_of(lens), Hv // Hk

    def run(t):
        end = torch.empty_like(t[5])
        return rule(*t[:5], offsets=off, state_in=t[5], state_out=end), end

    clean, clean_end = run([up(t) for t in data])
    assert torch.isfinite(clean).all()
    # first and last token of a chunk, inside a tile of 16, in the second chunk
    for t in {chunk_first, chunk_first + 1, chunk_first + 21, min(chunk_first + 63, lens[0] - 1)}:
        d = [x.clone() for x in data]
        h = 1 if d[names.index(name)].shape[1] > 1 else 0
        col = Dv - 1
        if name == "state":
            d[5][0, h, 3, col] = bad
            t = 0
        elif name in ("g", "beta"):
            d[names.index(name)][t, h] = bad
        else:
            d[names.index(name)][t, h, col if name == "v" else 3] = bad
        o, end = run([up(x) for x in d])
        hit = torch.zeros_like(o, dtype=torch.bool)
        heads = of_head(name, h, group)
        cols = slice(col, col + 1) if name in ("v", "state") else slice(0, Dv)
        hit[t:t + 1 if name == "q" else lens[0], heads, cols] = True
        assert torch.equal(o[~hit], clean[~hit]), (t, "an output that must not see it changed")
        assert not torch.isfinite(o[hit]).any(), (t, "an output that must show it is a number")
        ends = torch.zeros_like(end, dtype=torch.bool)
        if name != "q":
            ends[0, heads, :, cols] = True
        assert torch.equal(end[~ends], clean_end[~ends]) and not torch.isfinite(end[ends]).any()


# ---------------------------------------------------------------------------
# activations far from zero
# ---------------------------------------------------------------------------
def far_values(n):
    """fp32 values from -85 to 85 (their sigmoids are normal fp32 numbers), and the
    two signs of zero."""
    z = torch.linspace(-85, 85, n - 2, dtype=torch.float64) + 0.37 * torch.sin(torch.arange(n - 2, dtype=torch.float64))
    return torch.cat([z.clamp(-85, 85), torch.tensor([0.0, -0.0], dtype=torch.float64)]).float()


def within(got, want, tol, what):
    bad = (got.double().cpu() - want).abs() > tol
    i = int((((got.double().cpu() - want).abs() / tol.clamp_min(1e-300))).argmax())
    print(f"{what}: worst {float((got.double().cpu() - want).abs().flatten()[i] / tol.flatten()[i]):.2f} of the bound", flush=True)
    assert not bad.any(), what


# e^-|z| is off by an instruction of one unit in the last place (2 U) and two
# roundings, 1 + e^-|z| by one, the reciprocal by 2 U and a product by one: 8 U
# relative for the sigmoid and for its distance to 1, rounded up to 10; silu is a
# product more: 12.  The slope p (1 + z q) has 10 U of p, 10 of q, two products and
# a sum: 24 U of p (1 + |z| q).
SIG, SILU, SLOPE = 10 * ref.U, 12 * ref.U, 24 * ref.U


def test_silu_of_far_values_in_the_convolution():
    C, T = 64, 4096
    z = far_values(C * T).view(T, C)
    conv = dw.CausalDepthwiseConv1d(C, 2, "f32", act="silu")
    w = torch.stack([torch.zeros(C), torch.ones(C)])  # z is x itself
    p, q = torch.sigmoid(z.double()), torch.sigmoid(-z.double())
    want, slope = z.double() * p, p * (1 + z.double() * q)
    y = conv(up(z), up(w))
    within(y, want, SILU * want.abs(), "forward")
    state = torch.zeros(T, 1, C, device=DEV)
    within(conv.step(up(z), up(w), None, state=state), want, SILU * want.abs(), "step")
    dx, _, _, _ = conv.backward(up(z), up(w), torch.ones(T, C, device=DEV))
    within(dx, slope, SLOPE * p * (1 + z.double().abs() * q), "slope")
    special = torch.tensor([[INF, NAN, -INF, -200.0, 200.0, -1e30, 0.0, -0.0]])
    got = dw.CausalDepthwiseConv1d(8, 2, "f32", act="silu")(up(special), up(w[:, :8].contiguous()))[0].cpu()
    assert got[0] == INF and got[1:3].isnan().all() and (got[[3, 5, 6, 7]] == 0).all() and got[4] == 200.0


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("per", [1, 3])
def test_gates_of_far_values(act, per):
    D, rows = 96, 3000
    gate = far_values(D * -(-rows // per)).view(-1, D)
    norm = dw.BlockNorm(D, "f32", after="none", before="none", gate_act=act)
    one = torch.ones(rows, D, device=DEV)
    z = gate.double()
    p, q = torch.sigmoid(z), torch.sigmoid(-z)
    want = p if act == "sigmoid" else z * p
    h, _ = norm(one, gate=up(gate), rows_per_gate=per)
    spread = lambda t: t.repeat_interleave(per, 0)[:rows]  # noqa: E731
    within(h, spread(want), spread((SIG if act == "sigmoid" else SILU) * want.abs()), act)
    dgate = norm.backward(one, one, gate=up(gate), rows_per_gate=per)[2]
    # per equal terms are added: two roundings more
    slope, size = (p * q, p * q) if act == "sigmoid" else (p * (1 + z * q), p * (1 + z.abs() * q))
    within(dgate, per * slope, (SLOPE + per * ref.U) * per * size, act + " slope")
    special = torch.tensor([[INF, NAN, -INF, -200.0, 200.0, -1e30, 0.0, -0.0]])
    small = dw.BlockNorm(8, "f32", after="none", before="none", gate_act=act)
    got = small(torch.ones(1, 8, device=DEV), gate=up(special))[0][0].cpu()
    assert got[1].isnan()
    if act == "sigmoid":
        assert got[0] == 1 and got[2] == 0 and got[3] == 0 and got[4] == 1 and got[5] == 0 and (got[6:] == 0.5).all()
    else:
        assert got[0] == INF and got[2].isnan() and (got[[3, 5, 6, 7]] == 0).all() and got[4] == 200.0


# ---------------------------------------------------------------------------
# a given stream
# ---------------------------------------------------------------------------
CALLS = {
    "causal forward": lambda: (dw.CausalDepthwiseConv1d(256, 4, "f32"), lambda p, t, **k: p(*t, **k),
                                  lambda r: [r(300, 256), r(4, 256), r(256)]),
    "causal step": lambda: (dw.CausalDepthwiseConv1d(256, 4, "f32"), lambda p, t, **k: p.step(*t, **k),
                               lambda r: [r(300, 256), r(4, 256), r(256), r(300, 3, 256)]),
    "causal backward": lambda: (dw.CausalDepthwiseConv1d(256, 4, "f32"), lambda p, t, **k: p.backward(*t, **k),
                                   lambda r: [r(300, 256), r(4, 256), r(300, 256), r(256)]),
    "delta forward": lambda: (dw.GatedDeltaRule(1, 2, 64, 64, "f32"), lambda p, t, **k: p(*t, **k),
                                 lambda r: [r(300, 1, 64), r(300, 1, 64), r(300, 2, 64), -r(300, 2).abs(), r(300, 2)]),
    "delta step": lambda: (dw.GatedDeltaRule(1, 2, 64, 64, "f32"), lambda p, t, **k: p.step(*t, **k),
                              lambda r: [r(30, 1, 64), r(30, 1, 64), r(30, 2, 64), -r(30, 2).abs(), r(30, 2),
                                         r(30, 2, 64, 64)]),
    "delta backward": lambda: (dw.GatedDeltaRule(1, 2, 64, 64, "f32"), lambda p, t, **k: p.backward(*t, **k),
                                  lambda r: [r(300, 1, 64), r(300, 1, 64), r(300, 2, 64), -r(300, 2).abs(), r(300, 2),
                                             r(300, 2, 64)]),
    "norm forward": lambda: (dw.BlockNorm(256, "f32"), lambda p, t, **k: p(t[0], t[1], t[2], None, t[3], None, t[4], **k),
                                lambda r: [r(300, 256), r(300, 256), r(300, 256), r(256), r(256)]),
    "norm backward": lambda: (dw.BlockNorm(256, "f32"),
                                 lambda p, t, **k: p.backward(t[0], t[1], t[2], t[3], t[4], None, t[5], None, t[6], **k),
                                 lambda r: [r(300, 256) for _ in range(5)] + [r(256), r(256)]),
}


@pytest.mark.parametrize("name", CALLS)
def test_inputs_dropped_after_a_call_on_another_stream(name):
    """Memory of inputs that are dropped while the call still waits on its stream is
    not given to another tensor before the call has read it."""
    say(f"[gpu] dropped inputs: {name}")
    plan, call, make = CALLS[name]()
    seeds = iter(range(100))
    data = make(lambda *shape: rand(*shape, seed=next(seeds)) * 0.3)
    want = call(plan, [up(t) for t in data])
    want = [t.clone() for t in (want if isinstance(want, tuple) else (want,)) if t is not None]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    mine = [up(t) for t in data]
    taken = {t.data_ptr() for t in mine}
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)
    got = call(plan, mine, stream=side)
    del mine
    others = [torch.full(t.shape, NAN, device=DEV) for t in data for _ in range(2)]  # (nothing here waits for a stream)
    waiting = not side.query()
    print(f"{name}: {'still waiting' if waiting else 'already run'}", flush=True)
    assert not waiting or not taken & {t.data_ptr() for t in others}, "the memory of a dropped input is in use"
    torch.cuda.synchronize()
    got = [t for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------
# autograd
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("name", CALLS)
def test_a_tensor_that_requires_a_gradient_is_refused(name):
    """Whichever input it is; without gradients enabled it is taken."""
    plan, call, make = CALLS[name]()
    data = [up(t) for t in make(lambda *shape: rand(*shape) * 0.3)]
    for i in range(len(data)):
        d = [t.detach().clone().requires_grad_(j == i) for j, t in enumerate(data)]
        with pytest.raises(ValueError, match="autograd"):
            call(plan, d)
        with torch.no_grad():
            call(plan, d)


def test_the_operators_in_an_autograd_function():
    """How a training step has them: forward and backward as a Function's."""
    conv = dw.CausalDepthwiseConv1d(64, 4, "f32")

    class Mix(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            ctx.save_for_backward(x, w, b)
            return conv(x, w, b)

        @staticmethod
        def backward(ctx, dy):
            x, w, b = ctx.saved_tensors
            return conv.backward(x, w, dy.contiguous(), b)[:3]

    x, w, b = (up(rand(*s)).requires_grad_() for s in ((50, 64), (4, 64), (64,)))
    (Mix.apply(x, w, b) * 3).sum().backward()
    with torch.no_grad():
        want = conv.backward(x, w, torch.full_like(x, 3.0), b)
    assert all(torch.equal(t.grad, g) for t, g in zip((x, w, b), want))


# ---------------------------------------------------------------------------
# keys and queries of length zero
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt,Hk,Hv,Dk,Dv,lens,state", [
    ("f32", 1, 2, 40, 24, [70, 20], True), ("bf16", 1, 2, 128, 48, [130], False), ("f16", 2, 4, 64, 33, [65, 1, 90], True),
    ("bf16", 1, 1, 200, 40, [100], True), ("f16", 1, 3, 250, 16, [64, 30], True),
], ids=str)
def test_delta_gradients_at_zero_keys_and_queries(fmt, Hk, Hv, Dk, Dv, lens, state):
    """|x| = sqrt(sum x^2 + eps) has a slope at zero: the gradient of the unit vector
    over sqrt(eps), a thousand times it.  So is its error: the bounds of the other
    rows (tests/test_gpu_seq.py), times that for these."""
    say(f"[gpu] delta zero keys {fmt} {Hk} {Hv} {Dk} {Dv} {lens}")
    q, k, v, g, beta, s = delta_data(fmt, Hk, Hv, Dk, Dv, lens, state, gates="plain", seed=90)
    T, eps = sum(lens), 1e-6
    k[1::9], q[2::7], k[5::31], q[5::31] = 0.0, 0.0, 0.0, 0.0
    do = rand(T, Hv, Dv, seed=50, dtype=fmt)
    dso = rand(len(lens), Hv, Dk, Dv, seed=51, std=0.3) if state else None
    got = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, fmt, eps=eps).backward(*(up(t) for t in (q, k, v, g, beta, do)),
                                                                    offsets=offsets_of(lens), state_in=up(s), dstate_out=up(dso))
    args = leaves(q, k, v, g, beta, s)
    o, states, size = ref.delta(*args[:5], lens, args[5], Dk ** -0.5, True, eps)
    outs, gives, wrt = ([o, states], [do.double(), dso.double()], args) if state else ([o], [do.double()], args[:5])
    want = torch.autograd.grad(outs, wrt, gives)
    half, n = ref.HALF[q.dtype], Dk + 64 + Dv
    for name, i, x in (("dq", 0, q), ("dk", 1, k)):
        a, w, zero = got[i].double().cpu(), want[i], x.double().abs().sum(-1) == 0
        assert zero.any() and not zero.all()
        for rows, lift in ((zero, eps ** -0.5), (~zero, 1.0)):
            top = float(w[rows].abs().max()) / lift + float(w[~zero].abs().max()) + size
            off = (a[rows] - w[rows]).abs()
            assert (off <= half * w[rows].abs() + 8 * n * ref.U * top * lift).all(), (name, lift, float(off.max()))
            many = 24 * n ** 0.5 * ref.U * top * lift * w[rows].numel() ** 0.5
            assert float(off.norm()) <= half * float(w[rows].norm()) + many, (name, lift)
    for name, i in (("dv", 2), ("dg", 3), ("dbeta", 4)):
        assert rel(got[i].cpu(), want[i]) <= (half if i == 2 else 0) + 24 * n ** 0.5 * ref.U, name


# ---------------------------------------------------------------------------
# gradients of the convolution within bounds of their own size
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("case", CONV_GRADS, ids=lambda c: f"{c[0]}-C{c[1]}-K{c[2]}-{sum(c[3])}-{c[4]}")
def test_conv_gradients_to_the_sums_own_accuracy(case):
    """Element by element and in the 2-norm; the bounds see gradients that were summed
    or kept in fewer bits (tests/test_seq_bounds.py)."""
    say(f"[gpu] causal bwd, own accuracy {case}")
    x, w, b, s, dy, dso = conv_grad_data(case)
    fmt, C, K, lens, act, state = case
    got = dw.CausalDepthwiseConv1d(C, K, fmt, act=act).backward(
        up(x), up(w), up(dy), up(b), offsets=offsets_of(lens), state_in=up(s), dstate_out=up(dso))
    for name, g, (want, bound) in zip(("dx", "dw", "dbias", "dstate"), got, conv_grad_bounds(case, x, w, b, s, dy, dso)):
        if want is None:
            assert g is None
            continue
        off = (g.double().cpu() - want).abs()
        print(f"{name}: {float((off / bound).max()):.2f} of the bound, {float(off.norm() / bound.norm()):.2f} in the 2-norm", flush=True)
        assert (off <= bound).all() and float(off.norm()) <= 0.5 * float(bound.norm()), name


@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
def test_delta_gradient_through_a_large_exponent(fmt):
    """Sequences of two tokens whose second has g = 46 .. 85: its gradient is e^g times
    two dot products, of Dk and Dv positive products, so each relative error is the
    exponential's and the sums' rounding, sqrt(Dk + Dv) u, with 64 more for the
    products in between; e^g of a rounded g / ln 2 would be off by 25 u on average."""
    Dk, Dv, n = 64, 32, 128
    q, k, v, _, beta, _ = delta_data(fmt, 1, 1, Dk, Dv, [2] * n, False, gates="plain", seed=120)
    q, k, v, do = (t.abs() for t in (q, k, v, rand(2 * n, 1, Dv, seed=122, dtype=fmt)))
    g = torch.zeros(2 * n, 1)
    g[1::2, 0] = torch.linspace(46, 85, n)
    beta = beta.clamp_min(0.2)
    got = dw.GatedDeltaRule(1, 1, Dk, Dv, fmt).backward(*(up(t) for t in (q, k, v, g, beta, do)), offsets=offsets_of([2] * n))
    args = leaves(q, k, v, g, beta)
    o, _, _ = ref.delta(*args, [2] * n, None, Dk ** -0.5, True, 1e-6)
    want = torch.autograd.grad(o, args, do.double())[3][1::2]
    off = got[3].double().cpu()[1::2] / want - 1
    print(f"{fmt}: {float(off.norm()) / n ** 0.5 / ref.U:.1f} u on average", flush=True)
    assert float(off.norm()) / n ** 0.5 <= (Dk + 64 + Dv) ** 0.5 * ref.U


def test_more_sequences_than_2_to_the_30():
    """Nearly all of them empty: the search for a token's sequence passes sums of
    2^31, and the last sequence's tokens still find it."""
    C, K, n = 8, 3, 2 ** 30 + 5
    say("[gpu] 2^30 sequences")
    x, w = up(rand(9, C, seed=1)), up(rand(K, C, seed=2))
    off = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
    off[n - 1], off[n] = 4, 9  # the last two have tokens
    conv = dw.CausalDepthwiseConv1d(C, K, "f32")
    few = offsets_of([4, 5])
    assert torch.equal(conv(x, w, offsets=off), conv(x, w, offsets=few))
    a, b = (conv.backward(x, w, x, offsets=o) for o in (off, few))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    del off
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt,C,K", [("bf16", 64, 4), ("f32", 9, 3)])
def test_many_empty_sequences_between_tokens(fmt, C, K):
    """A border in the middle of a run with 2^26 empty sequences on it is passed in a
    search, not one by one."""
    say(f"[gpu] empty sequences {fmt}")
    lens, n = [5, 30, 1, 20], 2 ** 26
    x, w, dy = up(rand(60, C, seed=1, dtype=fmt)), up(rand(K, C, seed=2, dtype=fmt)), up(rand(60, C, seed=3, dtype=fmt))
    conv, few = dw.CausalDepthwiseConv1d(C, K, fmt), offsets_of(lens)
    off = torch.full((3 * n + 5,), 5, dtype=torch.int32, device=DEV)
    off[0], off[n + 2:2 * n + 3], off[2 * n + 3:3 * n + 4], off[3 * n + 4] = 0, 35, 36, 56
    assert off.diff().min() >= 0 and (off.diff() > 0).sum() == 4
    y, want = torch.full((60, C), 7.0, dtype=x.dtype, device=DEV), torch.full((60, C), 7.0, dtype=x.dtype, device=DEV)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    conv(x, w, offsets=few, y=want)
    start.record()
    conv(x, w, offsets=off, y=y)
    stop.record()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and start.elapsed_time(stop) < 100, start.elapsed_time(stop)
    dx, dxw = y.clone(), y.clone()
    a, b = (conv.backward(x, w, dy, offsets=o, dx=d) for o, d in ((off, dx), (few, dxw)))
    assert torch.equal(dx, dxw) and torch.equal(a[1], b[1])


def test_norm_without_a_second_norm_returns_no_second_output():
    o, w = up(rand(5, 64)), torch.ones(64, device=DEV)
    given = torch.full_like(o, 7.0)
    h, y = dw.BlockNorm(64, "f32", before="none")(o, w_after=w, y=given)
    assert y is None and (given == 7.0).all() and torch.isfinite(h).all()


def test_captured_with_a_given_stream():
    """Passes captured on the stream that they are given, inputs dropped inside the
    capture, replayed between eager ones."""
    conv, rule = dw.CausalDepthwiseConv1d(192, 4, "bf16"), dw.GatedDeltaRule(1, 1, 64, 64, "bf16")
    x, w, b = up(rand(130, 192, seed=1, dtype="bf16")), up(rand(4, 192, seed=2, dtype="bf16")), up(rand(192, seed=3))
    g, beta = -up(rand(130, 1, seed=4)).abs(), torch.sigmoid(up(rand(130, 1, seed=5)))

    def passes(stream):
        mixed = conv(x * 2, w, b, stream=stream)
        q, k, v = (t.unflatten(1, (1, 64)) for t in mixed.split([64, 64, 64], 1))
        o = rule(q, k, v, g, beta, stream=stream)
        del mixed, q, k, v
        return o, conv.backward(x * 3, w, x * 5, b, stream=stream)[1]

    want = [t.clone() for t in passes(None)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = passes(torch.cuda.current_stream())
    for _ in range(3):
        for t in got:
            t.fill_(-7)
        eager = passes(None)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(got, want, eager))
    del graph


@pytest.mark.parametrize("case", [("bf16", 4, 8, 128, 128, 140), ("f16", 2, 16, 200, 48, 66), ("f32", 1, 4, 30, 68, 300)],
                         ids=lambda c: "-".join(map(str, c)))
def test_delta_steps_of_many_heads(case):
    """More than 1024 heads of all rows together."""
    test_gpu_seq.test_delta_steps_follow_the_definition(case)
