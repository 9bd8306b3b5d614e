"""The selective scan and the group norm on the GPU where tests/test_gpu_scan.py does not
reach: states that grow, long runs, every number of lanes a channel, wide slices, streams."""
import pytest
import torch

import depthwise_convolution_amd as dw
import scan_reference as ref
from gpu_helpers import DEV, say
from seq_reference import U, leaves

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
