"""The selective scan of one long sequence in 64 bits: the values and bounds of
tests/scan_reference.py's ``scan_bounds`` for all tokens at once instead of one by one.

Each of its recurrences is h_t = e_t h_(t-1) + put_t, which ``linear`` forms in blocks: every
block from zero, side by side, and the blocks one after the other by the product of their e.
(tests/test_scan_long_reference.py holds the two forms against each other.)"""
import torch

from scan_cases import scan_data
from scan_reference import LEAST, act_of, slope_of, softplus
from seq_reference import HALF, U


def linear(e, put, first):
    """All h_t of h_t = e_t h_(t-1) + put_t, h before the first token ``first``."""
    T = put.shape[0]
    L = max(1, int(T ** 0.5))
    n = -(-T // L)
    pad = n * L - T
    if pad:
        e = torch.cat([e, torch.ones_like(e[:1]).expand(pad, *e.shape[1:])])
        put = torch.cat([put, torch.zeros_like(put[:1]).expand(pad, *put.shape[1:])])
    e, put = e.reshape(n, L, *e.shape[1:]), put.reshape(n, L, *put.shape[1:])
    h, fade = torch.empty_like(put), torch.empty_like(put)
    s, p = torch.zeros_like(put[:, 0]), torch.ones_like(put[:, 0])
    for j in range(L):
        s, p = e[:, j] * s + put[:, j], p * e[:, j]
        h[:, j], fade[:, j] = s, p
    start = torch.empty_like(s)
    for k in range(n):
        start[k] = first if k == 0 else fade[k - 1, -1] * start[k - 1] + h[k - 1, -1]
    h += fade * start[:, None]
    return h.reshape(n * L, *h.shape[2:])[:T]


def before(h, first):
    """h_(t-1) of every token."""
    return torch.cat([first[None], h[:-1]])


def back_linear(e, put, last):
    """All g_t of g_t = e_(t+1) g_(t+1) + put_t, e_(t+1) g_(t+1) behind the last token ``last``."""
    one = torch.ones_like(e[:1])
    return linear(torch.cat([one, e[1:].flip(0)]), put.flip(0), last).flip(0)


def long_bounds(dtype, x, dt, a, b, c, skip, bias, gate, state, soft=True, act="silu", dy=None, dstate=None, terms=None):
    """As ``scan_bounds`` of one sequence; sums over tokens go through chains of at most
    ``terms`` additions (None: all tokens)."""
    half, least = HALF[dtype], LEAST[dtype]
    f = lambda t: None if t is None else t.double()  # noqa: E731
    x, dt, a, b, c, skip, bias, gate, state, dy, dstate = (f(t) for t in (x, dt, a, b, c, skip, bias, gate, state, dy, dstate))
    (C, N), G, T = a.shape, b.shape[1], x.shape[0]
    terms = T if terms is None else terms
    grow = lambda t: t.repeat_interleave(C // G, 1)  # noqa: E731
    fold = lambda t: t.view(T, G, C // G, N).sum(2)  # noqa: E731
    v = dt if bias is None else dt + bias
    d, sl = (softplus(v), torch.sigmoid(v)) if soft else (v, torch.ones_like(v))
    ed = ((2 * v.abs() + 8) if soft else torch.ones_like(v)) * U
    z = torch.zeros_like(x) if gate is None else gate
    gv, gs = (act_of(z, act), slope_of(z, act)) if gate is not None else (torch.ones_like(z), torch.zeros_like(z))
    eg = (z.abs() + 8) * U * gv.abs() if gate is not None else torch.zeros_like(z)
    egs = 2 * (z.abs() + 8) * (1 + z.abs()) * U if gate is not None else torch.zeros_like(z)
    sk = torch.zeros(C, dtype=torch.float64) if skip is None else skip
    first = torch.zeros(C, N, dtype=torch.float64) if state is None else state
    none = torch.zeros_like(first)
    wide = lambda t: t[:, :, None]  # noqa: E731
    bt, ct = grow(b), grow(c)
    decay = torch.exp(wide(d) * a)
    ee = (wide(d) * a).abs() * (wide(ed) + 2 * U) + 2 * U
    put = wide(d * x) * bt
    eput = (wide(ed) + 4 * U) * put.abs()
    h, M = linear(decay, put, first), linear(decay, put.abs(), first.abs())
    h0, M0 = before(h, first), before(M, first.abs())
    E = linear(decay, (ee + 2 * U) * decay * M0 + eput, none)
    top = torch.maximum(M.cummax(0).values, first.abs())
    yp = (h * ct).sum(2) + sk * x
    ype = ((E + 100 * U * top + (N + 2) * U * M) * ct.abs()).sum(2) + 3 * U * (sk * x).abs()
    y = yp * gv
    ye = gv.abs() * ype + (eg + 2 * U * gv.abs()) * yp.abs() + half * y.abs() + least
    fin = h[-1]
    out = {"y": (y, ye), "state": (fin[None], (E[-1] + 100 * U * top[-1] + U * fin.abs())[None])}
    if dy is None:
        return out
    stored = lambda t, e: (t, e + half * t.abs() + least)  # noqa: E731
    E0 = before(E, none) + 100 * U * top[-1]
    E1 = decay * E0 + (ee + 2 * U) * decay * M0 + eput
    dyt = dy * gv
    edy = dy.abs() * eg + U * dyt.abs()
    if gate is not None:
        dgate = dy * yp * gs
        out["dgate"] = stored(dgate, dy.abs() * (ype * gs.abs() + yp.abs() * egs) + 3 * U * dgate.abs())
    out["dskip"] = ((dyt * x).sum(0), ((edy + (terms + 2) * U * dyt.abs()) * x.abs()).sum(0))
    out["dc"] = stored(fold(wide(dyt) * h), fold(wide(dyt.abs()) * (E1 + (C // G + 2) * U * M) + wide(edy) * M))
    last = none if dstate is None else dstate
    cd = ct * wide(dyt)
    D, MD = back_linear(decay, cd, last), back_linear(decay, cd.abs(), last.abs())
    was = MD - cd.abs()
    more = ct.abs() * wide(edy) + U * (was + 2 * cd.abs())
    lost = (ee + 2 * U) * decay * MD  # of G e, for the token before
    ED = back_linear(decay, more + torch.cat([lost[1:], torch.zeros_like(lost[:1])]), none)
    topd = torch.maximum(MD.flip(0).cummax(0).values.flip(0), last.abs())
    EDj = ED + 100 * U * topd
    out["db"] = stored(fold(D * wide(d * x)), fold(wide((d * x).abs()) * (EDj + (wide(ed) + (C // G + 3) * U) * MD)))
    du, Mdu = (D * bt).sum(2), (MD * bt.abs()).sum(2)
    Edu = (bt.abs() * (EDj + (N + 1) * U * MD)).sum(2)
    out["dx"] = stored(du * d + sk * dyt, d.abs() * (Edu + (ed + 2 * U) * Mdu) + sk.abs() * (edy + 2 * U * dyt.abs()))
    through, Mt = D * decay * h0, MD * decay * M0
    Et = decay * (EDj * M0 + MD * E0) + (ee + 3 * U) * Mt
    dd, Mdd = (through * a).sum(2) + du * x, (Mt * a.abs()).sum(2) + Mdu * x.abs()
    Edd = ((Et + (N + 4) * U * Mt) * a.abs()).sum(2) + x.abs() * Edu + 3 * U * Mdd
    ddt, eddt = dd * sl, sl * (Edd + (ed + 2 * U) * Mdd)
    out["ddt"] = stored(ddt, eddt)
    out["dbias"] = (ddt.sum(0), (eddt + (terms + 2) * U * sl * Mdd).sum(0))
    out["da"] = ((wide(d) * through).sum(0), (wide(d.abs()) * (Et + (wide(ed) + (terms + 3) * U) * Mt)).sum(0))
    D0, MD0 = decay[0] * D[0], decay[0] * MD[0]
    ED0 = decay[0] * ED[0] + lost[0]
    out["dstate"] = (D0[None], (ED0 + 100 * U * topd[0])[None])
    return out


# fmt, channels, states, groups, tokens of each sequence, gate activation, tokens a run (the
# fewest that fill the card: forward and gradients)
LONG = [
    ("f32", 3, 2, 1, [1600000], "silu", 1024),
    ("f16", 2, 3, 1, [800000, 6000], "sigmoid", 512),
    ("bf16", 2, 20, 1, [400000], "silu", 256),
    ("f16", 1, 40, 1, [200007], "silu", 128),
]


def long_id(c):
    return f"{c[0]}-C{c[1]}-N{c[2]}-{sum(c[4])}"


def long_data(case):
    fmt, C, N, G, lens, act, _ = case
    d = scan_data((fmt, C, N, G, lens, True, act, True, True, 0), seed=1)
    d["a"][:, ::2] /= 64
    return {k: v.abs() if k in ("x", "b", "c", "skip", "state", "dy", "dstate") else v for k, v in d.items()}
