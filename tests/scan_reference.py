"""Plain 64-bit forms of the selective scan and the group norm on the CPU,
written from the definitions in include/dwconv_seq.h, and bounds of what fp32
arithmetic may leave.

``scan`` and ``group`` are differentiable.  ``scan_bounds`` and ``group_bounds``
return {name: (value, bound of its error)}: values by the explicit recurrences
(held against autograd's and against differences in
tests/test_scan_reference.py), bounds by the same recurrences over magnitudes.
u is one fp32 rounding, 2^-24.

Scan.  v = dt + bias is off by u |v|, and e^-|v| by its rounded exponent, |v| u
(16-bit data), so the width d = softplus(v) and its slope by (2 |v| + 8) u of
themselves (slope / d and slope |v| / d are at most 1 where v < 0, resp. > 0).  A
decay e^(d a) takes that times |d a|, two more roundings of the exponent and
two of the instruction.  A state's error follows the state: E_t = e E_(t-1) plus
what the decay and a rounding leave of e M_(t-1), plus that of the input, M the
same recurrence over magnitudes.  Where runs of tokens are joined, their decay is
taken from the sum of up to 1024 widths, each lane's 256 of them one by one: 256 u
|a sum d| e^-|a sum d| <= 100 u of the state before: 100 u of the largest magnitude
of the sequence.  Gradients the same with the recurrence run backwards.  Sums over
states, channels and tokens of n terms take n u of their magnitudes.  The sigmoid of
the gate and its slope: (|z| + 8) u and 2 (|z| + 8) (1 + |z|) u.

What is stored is off by half a step: HALF of the value, and below the least normal
number half of the steps there, 2^-25 for fp16 (LEAST).

Group norm.  Sums over a group go through chains of at most 128 additions (vectors
of a lane, lanes of a workgroup, channels, runs): the mean is off by 128 u of the
mean magnitude (dm), the squares around it by 132 u and dm^2 / var, r by half of
that and three roundings.
"""
import torch

from seq_reference import HALF, U, starts


# half a step between the numbers next to zero (those of bf16 and fp32 are beyond any value here)
LEAST = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 0.0}


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def act_of(z, act):
    return z if act == "none" else torch.sigmoid(z) if act == "sigmoid" else z * torch.sigmoid(z) if act == "silu" \
        else z.clamp_min(0)


def slope_of(z, act):
    p, q = torch.sigmoid(z), torch.sigmoid(-z)
    return torch.ones_like(z) if act == "none" else p * q if act == "sigmoid" else p * (1 + z * q) if act == "silu" \
        else (z > 0).double()


def scan(x, dt, a, b, c, skip, bias, gate, lens, state, soft=True, act="silu"):
    """(y, final states); every tensor float64, tokens x ..., b and c tokens x G x N."""
    C, N = a.shape
    G = b.shape[1]
    grow = lambda t: t.repeat_interleave(C // G, 0)  # noqa: E731
    v = dt if bias is None else dt + bias
    d = softplus(v) if soft else v
    ys, finals = [], []
    for i, (s, n) in enumerate(zip(starts(lens), lens)):
        h = x.new_zeros(C, N) if state is None else state[i]
        for t in range(s, s + n):
            h = torch.exp(d[t][:, None] * a) * h + (d[t] * x[t])[:, None] * grow(b[t])
            y = (h * grow(c[t])).sum(1)
            y = y if skip is None else y + skip * x[t]
            ys.append(y if gate is None else y * act_of(gate[t], act))
        finals.append(h)
    return torch.stack(ys) if ys else x.new_zeros(0, C), torch.stack(finals) if finals else x.new_zeros(0, C, N)


def scan_bounds(dtype, x, dt, a, b, c, skip, bias, gate, lens, state, soft=True, act="silu", dy=None, dstate=None):
    """{y, state} and, with dy, {dx, ddt, da, db, dc, dskip, dbias, dgate, dstate}: (value, bound)."""
    half, least = HALF[dtype], LEAST[dtype]
    f = lambda t: None if t is None else t.double()  # noqa: E731
    x, dt, a, b, c, skip, bias, gate, state, dy, dstate = (f(t) for t in (x, dt, a, b, c, skip, bias, gate, state, dy, dstate))
    (C, N), G, T = a.shape, b.shape[1], sum(lens)
    grow = lambda t: t.repeat_interleave(C // G, 0)  # noqa: E731
    fold = lambda t: t.view(G, C // G, N).sum(1)  # noqa: E731
    v = dt if bias is None else dt + bias
    d, sl = (softplus(v), torch.sigmoid(v)) if soft else (v, torch.ones_like(v))
    ed = ((2 * v.abs() + 8) if soft else torch.ones_like(v)) * U  # relative error of d and of its slope
    z = torch.zeros_like(x) if gate is None else gate
    gv, gs = (act_of(z, act), slope_of(z, act)) if gate is not None else (torch.ones_like(z), torch.zeros_like(z))
    eg = (z.abs() + 8) * U * gv.abs() if gate is not None else torch.zeros_like(z)
    egs = 2 * (z.abs() + 8) * (1 + z.abs()) * U if gate is not None else torch.zeros_like(z)
    sk = torch.zeros(C, dtype=torch.float64) if skip is None else skip
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    y, ye, yp, ype = zero(T, C), zero(T, C), zero(T, C), zero(T, C)
    fin, fine = zero(len(lens), C, N), zero(len(lens), C, N)
    g = {k: zero(*s) for k, s in dict(dx=(T, C), ddt=(T, C), da=(C, N), db=(T, G, N), dc=(T, G, N), dskip=(C,), dbias=(C,),
                                      dgate=(T, C), dstate=(len(lens), C, N)).items()}
    e = {k: torch.zeros_like(t) for k, t in g.items()}
    for i, (s, n) in enumerate(zip(starts(lens), lens)):
        h = zero(C, N) if state is None else state[i]
        M, E, kept = h.abs(), zero(C, N), []
        top = M.clone()
        for t in range(s, s + n):
            decay = torch.exp(d[t][:, None] * a)
            ee = (d[t][:, None] * a).abs() * (ed[t][:, None] + 2 * U) + 2 * U  # relative
            put = (d[t] * x[t])[:, None] * grow(b[t])
            kept.append((h, M, E, decay, ee))
            E = decay * E + (ee + 2 * U) * decay * M + (ed[t][:, None] + 4 * U) * put.abs()
            h, M = decay * h + put, decay * M + put.abs()
            top = torch.maximum(top, M)
            ct = grow(c[t])
            yp[t] = (h * ct).sum(1) + sk * x[t]
            ype[t] = ((E + 100 * U * top + (N + 2) * U * M) * ct.abs()).sum(1) + 3 * U * (sk * x[t]).abs()
            y[t] = yp[t] * gv[t]
            ye[t] = gv[t].abs() * ype[t] + (eg[t] + 2 * U * gv[t].abs()) * yp[t].abs() + half * y[t].abs() + least
        fin[i], fine[i] = h, E + 100 * U * top
        if dy is None:
            continue
        D = zero(C, N) if dstate is None else dstate[i]
        MD, ED = D.abs(), zero(C, N)
        topd = MD.clone()
        for t in range(s + n - 1, s - 1, -1):
            h0, M0, E0, decay, ee = kept[t - s]
            E0 = E0 + 100 * U * top
            dt_, xt, et = d[t][:, None], x[t][:, None], ed[t][:, None]
            bt, ct = grow(b[t]), grow(c[t])
            h1 = decay * h0 + dt_ * xt * bt
            M1 = decay * M0 + (dt_ * xt * bt).abs()
            E1 = decay * E0 + (ee + 2 * U) * decay * M0 + (et + 4 * U) * (dt_ * xt * bt).abs()
            dyt = dy[t] * gv[t]
            edy = dy[t].abs() * eg[t] + U * dyt.abs()
            if gate is not None:
                g["dgate"][t] = dy[t] * yp[t] * gs[t]
                e["dgate"][t] = dy[t].abs() * (ype[t] * gs[t].abs() + yp[t].abs() * egs[t]) + (3 * U + half) * g["dgate"][t].abs() + least
            g["dskip"] += dyt * x[t]
            e["dskip"] += (edy + (T + 2) * U * dyt.abs()) * x[t].abs()
            g["dc"][t] = fold(dyt[:, None] * h1)
            e["dc"][t] = fold(dyt.abs()[:, None] * (E1 + (C // G + 2) * U * M1) + edy[:, None] * M1) + half * g["dc"][t].abs() + least
            ED = ED + ct.abs() * edy[:, None] + U * (MD + 2 * (ct * dyt[:, None]).abs())
            D, MD = D + ct * dyt[:, None], MD + (ct * dyt[:, None]).abs()
            topd = torch.maximum(topd, MD)
            EDj = ED + 100 * U * topd
            g["db"][t] = fold(D * dt_ * xt)
            e["db"][t] = fold((dt_ * xt).abs() * (EDj + (et + (C // G + 3) * U) * MD)) + half * g["db"][t].abs() + least
            du = (D * bt).sum(1)
            Mdu = (MD * bt.abs()).sum(1)
            Edu = (bt.abs() * (EDj + (N + 1) * U * MD)).sum(1)
            g["dx"][t] = du * d[t] + sk * dyt
            e["dx"][t] = d[t].abs() * (Edu + (ed[t] + 2 * U) * Mdu) + sk.abs() * (edy + 2 * U * dyt.abs()) + half * g["dx"][t].abs() + least
            through = D * decay * h0
            Mt = MD * decay * M0
            Et = decay * (EDj * M0 + MD * E0) + (ee + 3 * U) * Mt
            dd = (through * a).sum(1) + du * x[t]
            Mdd = (Mt * a.abs()).sum(1) + Mdu * x[t].abs()
            Edd = ((Et + (N + 4) * U * Mt) * a.abs()).sum(1) + x[t].abs() * Edu + 3 * U * Mdd
            g["ddt"][t] = dd * sl[t]
            more = sl[t] * (Edd + (ed[t] + 2 * U) * Mdd)
            e["ddt"][t] = more + half * g["ddt"][t].abs() + least
            g["dbias"] += g["ddt"][t]
            e["dbias"] += more + (T + 2) * U * sl[t] * Mdd
            g["da"] += dt_ * through
            e["da"] += dt_.abs() * (Et + (et + (T + 3) * U) * Mt)
            ED = decay * ED + (ee + 2 * U) * decay * MD
            D, MD = decay * D, decay * MD
        g["dstate"][i], e["dstate"][i] = D, ED + 100 * U * topd
    out = {"y": (y, ye), "state": (fin, fine + U * fin.abs())}
    if dy is not None:
        out.update({k: (g[k], e[k]) for k in g})
    return out


def group(x, w, b, G, act, eps):
    """y of images x pixels x C, float64."""
    n, S, C = x.shape
    v = x.view(n, S, G, C // G)
    v = v - v.mean((1, 3), keepdim=True)
    u = (v / torch.sqrt((v * v).mean((1, 3), keepdim=True) + eps)).view(n, S, C)
    z = u if w is None else u * w
    return act_of(z if b is None else z + b, act)


def group_bounds(dtype, x, w, b, G, act, eps, dy=None):
    """{y} and, with dy, {dx, dw, db}: (value, bound); "border": the least |z| over its error."""
    half, least = HALF[dtype], LEAST[dtype]
    n, S, C = x.shape
    x = x.double()
    w = torch.ones(C, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(C, dtype=torch.float64) if b is None else b.double()
    split = lambda t: t.view(n, S, G, C // G)  # noqa: E731
    over = lambda t: split(t).mean((1, 3), keepdim=True).expand(n, S, G, C // G).reshape(n, S, C)  # noqa: E731
    m = over(x)
    var = over((x - m) ** 2)
    r = (var + eps) ** -0.5
    dm = 128 * U * over(x.abs())
    er = 70 * U + dm ** 2 / (2 * (var + eps)) + 3 * U
    u = (x - m) * r
    Eu = r * (dm + U * (x - m).abs()) + u.abs() * (er + 2 * U)
    z = u * w + b
    Ez = Eu * w.abs() + 3 * U * ((u * w).abs() + b.abs())
    y = act_of(z, act)
    ez = (z.abs() + 8) * (1 + z.abs()) * U if act == "silu" else 0.0
    out = {"y": (y, 1.1 * Ez + ez + half * y.abs() + least), "border": float((z.abs() / Ez).min()) if z.numel() else 1e9}
    if dy is None:
        return out
    dy = dy.double()
    sl = slope_of(z, act)
    dz = dy * sl
    Edz = dy.abs() * ((0.5 * Ez + 2 * ez) if act == "silu" else 0.0) + U * dz.abs()
    m1, m2 = over(dz * w), over(dz * w * u)
    E1 = over(w.abs() * Edz) + 130 * U * over((dz * w).abs())
    E2 = over(w.abs() * (Edz * u.abs() + dz.abs() * Eu)) + 132 * U * over((dz * w * u).abs())
    size = (dz * w).abs() + m1.abs() + (u * m2).abs()
    dx = r * (dz * w - m1 - u * m2)
    Edx = r * (w.abs() * Edz + E1 + u.abs() * E2 + Eu * m2.abs() + 4 * U * size) + r * (er + 2 * U) * size
    total = lambda t: t.sum((0, 1))  # noqa: E731
    out["dx"] = (dx, Edx + half * dx.abs() + least)
    out["dw"] = (total(dz * u), total(Edz * u.abs() + dz.abs() * Eu) + (130 + n) * U * total((dz * u).abs()))
    out["db"] = (total(dz), total(Edz) + (128 + n) * U * total(dz.abs()))
    return out


def outside(got, want, bound):
    """True where an element is off by more than its bound, or the 2-norm of 64 errors or
    more by 0.75 of the bounds'.  Rounding to the type alone, all significands next to 1,
    leaves uniform errors up to the bound: a mean square of 1/3 of the bound's, whose own
    deviation is sqrt(4/45) / (1/3) = 0.894 of it over the root of their number, so at
    most (1 + 4 x 0.112) / 3 = 0.69^2 for 64 and four deviations; what sums leave are worst
    cases of every rounding at once, and less."""
    off = (got.double().cpu() - want).abs()
    if not bool((off <= bound).all()):
        return True
    return off.numel() >= 64 and float(off.norm()) > 0.75 * float(bound.norm()) + 1e-300
