"""Plain 64-bit forms of the sequence operators on the CPU, one token at a
time, written from the definitions in include/dwconv_seq.h.  They take and
return torch float64 tensors and are differentiable, so that gradients of the
kernels are compared with autograd's of the definition (and those with
differences in tests/test_seq_reference.py).

Tolerances.  A stored value is off by at most half a step, eps / 2 relative
(HALF).  In front of that come fp32 sums.  u = 2^-24 is one fp32 rounding.
"""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def conv(x, w, bias, lens, state, act):
    """(y, final states, z, sum of |terms| of z) of tokens x C."""
    K, C = w.shape
    ys, states, zs, scales = [], [], [], []
    for i, (a, n) in enumerate(zip(starts(lens), lens)):
        old = x.new_zeros(K - 1, C) if state is None else state[i]
        ext = torch.cat([old, x[a:a + n]])
        for t in range(n):
            terms = w * ext[t:t + K]
            z = terms.sum(0) + (0 if bias is None else bias)
            zs.append(z)
            scales.append(terms.detach().abs().sum(0) + (0 if bias is None else bias.detach().abs()))
            ys.append(z / (1 + torch.exp(-z)) if act == "silu" else z)
        states.append(ext[n:])
    stack = lambda v: torch.stack(v) if v else x.new_zeros(0, C)  # noqa: E731
    return stack(ys), torch.stack(states), stack(zs).detach(), stack(scales)


def delta(q, k, v, g, beta, lens, state, scale, normalize, eps):
    """(o, final states, largest norm of a state or a value met)."""
    Hk, Hv = q.shape[1], v.shape[1]
    if normalize:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + eps)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + eps)
    q = (q * scale).repeat_interleave(Hv // Hk, 1)
    k = k.repeat_interleave(Hv // Hk, 1)
    out, finals, size = [], [], 0.0
    for i, (a, n) in enumerate(zip(starts(lens), lens)):
        S = q.new_zeros(Hv, q.shape[2], v.shape[2]) if state is None else state[i]
        size = max(size, float(S.detach().norm(dim=(1, 2)).max()))
        for t in range(a, a + n):
            S = S * torch.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - (S * k[t][:, :, None]).sum(1))
            S = S + k[t][:, :, None] * u[:, None, :]
            out.append((S * q[t][:, :, None]).sum(1))
            size = max(size, float(S.detach().norm(dim=(1, 2)).max()), float(v[t].detach().norm(dim=1).max()))
        finals.append(S)
    o = torch.stack(out) if out else v.new_zeros(0, Hv, v.shape[2])
    return o, torch.stack(finals), size


def normed(x, kind, w, b, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return x if b is None or kind != "layer" else x + b


def block(o, residual, gate, per, scale, w_after, b_after, w_before, b_before, after, before, act, eps):
    """(h, y or None); o, residual rows x D, gate ceil(rows / per) x D."""
    t = normed(o, after, w_after, b_after, eps)
    if gate is not None:
        row = torch.arange(o.shape[0]) // per
        g = gate[row]
        t = t * (g if act == "none" else torch.sigmoid(g) if act == "sigmoid" else g * torch.sigmoid(g))
    if scale is not None:
        t = t * scale
    h = t if residual is None else residual + t
    return h, (None if before == "none" else normed(h, before, w_before, b_before, eps))


def rel(x, ref):
    """2-norm of the difference over that of the reference."""
    d = float((x.double() - ref).norm())
    n = float(ref.norm())
    return d / n if n else (math.inf if d else 0.0)


def leaves(*tensors):
    return [None if t is None else t.detach().double().requires_grad_() for t in tensors]
