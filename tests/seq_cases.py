"""Inputs and bounds that the CPU and the GPU tests of the sequence operators'
numerics share; everything here is torch float64 on the CPU."""
import math

import torch

import seq_reference as ref
from seq_reference import HALF, U


def in_terms(x, n):
    """x as the sum of n bf16 terms, each the nearest of what the ones before leave."""
    out, left = torch.zeros_like(x), x.clone()
    for _ in range(n):
        t = left.float().to(torch.bfloat16).double()
        out, left = out + t, left - t
    return out


# ---------------------------------------------------------------------------
# The delta rule read back under its own key: with q = k, beta = 1 and no decay
# the state answers a token with the token's value, o_t = scale S_t^T k_t =
# scale v_t, as the difference of two terms of the size of c_t = scale S_{t-1}^T
# k_t.  With values far smaller than the state the rounding of o to its type
# says nothing, and what is left of the sums shows.
# ---------------------------------------------------------------------------
def readback(fmt, Hk, Hv, Dk, Dv, lens, seed=0):
    """(q, k, v, g, beta, state) of tests' types on the CPU."""
    dt = ref.DTYPES[fmt]
    g = torch.Generator().manual_seed(seed + Dk)
    T = sum(lens)
    k = (torch.randn(T, Hk, Dk, generator=g) + 0.2).to(dt)
    v = (torch.randn(T, Hv, Dv, generator=g) * {"f32": 2.0 ** -14, "f16": 2.0 ** -8, "bf16": 2.0 ** -12}[fmt]).to(dt)
    state = torch.randn(len(lens), Hv, Dk, Dv, generator=g) * 64
    return k.clone(), k, v, torch.zeros(T, Hv), torch.ones(T, Hv), state


def readback_terms(q, k, lens, state, v, scale, eps):
    """c_t of every token, the size of the two terms that cancel."""
    Hv = v.shape[1]
    q, k = (x.double() / torch.sqrt((x.double() ** 2).sum(-1, keepdim=True) + eps) for x in (q, k))
    q, k = (x.repeat_interleave(Hv // x.shape[1], 1) for x in (q * scale, k))
    out, at = [], 0
    for i, n in enumerate(lens):
        S = state[i].double()
        for t in range(at, at + n):
            out.append((S * q[t][:, :, None]).sum(1))
            S = S + k[t][:, :, None] * (v[t].double() - (S * k[t][:, :, None]).sum(1))[:, None, :]
        at += n
    return torch.stack(out)


def readback_bound(dt, want, c, Dk):
    """Largest 2-norm of o's error.  o is off by its rounding and by what two
    chained sums in fp32 (K S into U, then Q S + P U) of up to Dk + 64 products
    leave, sqrt(n) U of the size of what they add each: 2 sqrt(Dk + 64) U |c|."""
    return HALF[dt] * float(want.norm()) + 2 * math.sqrt(Dk + 64) * U * float(c.norm())


# ---------------------------------------------------------------------------
# Gradients of the causal convolution.  u is one fp32 rounding, s_t the sum of the
# magnitudes of z_t's terms:
#   z      (K + 1) u s_t;  silu's slope has |silu''| <= 0.5
#   slope  0.5 of z's error, and its own evaluation, where the sigmoid is off by
#          (|z| + 4) u of itself and one minus it by 2 u: 2 (|z| + 8) (1 + |z|) u
#   dz     |dy| times the slope's error and a product; exactly dy without silu
#   dx     the K terms' errors added, K u of their magnitudes, and its rounding;
#          dstate the same
#   dw     errors of independent roundings: 4 sqrt(sum (ext e_t)^2), and 2 sqrt(T) u
#          of sqrt(sum (ext dz)^2) for the sum itself; dbias the same with ext = 1;
#          u of the value for its rounding
# Worst cases all of them, so the 2-norm of the errors stays below half the bounds'.
# ---------------------------------------------------------------------------
CONV_GRADS = [  # fmt, C, K, lens, act, state
    ("f32", 1024, 4, [300, 1, 2, 3, 400], "silu", True), ("f32", 130, 2, [64, 65, 1], "none", True),
    ("bf16", 128, 8, [200, 3], "silu", True), ("bf16", 96, 3, [2500], "silu", False),
    ("f16", 61, 4, [5, 0, 2, 300], "silu", True), ("f16", 64, 6, [130, 500], "none", False),
    ("f32", 7, 5, [0, 0, 900], "silu", False), ("bf16", 1, 7, [400, 6], "silu", True),
]


def conv_grad_data(case):
    fmt, C, K, lens, act, state = case
    dt, T = ref.DTYPES[fmt], sum(lens)
    g = torch.Generator().manual_seed(C + 31 * K + T)
    r = lambda *shape: torch.randn(shape, generator=g)  # noqa: E731
    return (r(T, C).to(dt), (r(K, C) * K ** -0.5).to(dt), r(C) * 0.3, r(len(lens), K - 1, C).to(dt) if state else None,
            r(T, C).to(dt), r(len(lens), K - 1, C).to(dt) if state else None)


def conv_grad_bounds(case, x, w, b, s, dy, dso):
    """[(gradient in 64 bits, bound of its error)] of x, w, bias and the state."""
    fmt, C, K, lens, act, state = case
    half, T = HALF[x.dtype], sum(lens)
    W, B, at = w.double(), b.double(), 0
    dxs, dstates = [], []
    dw, dw_e, dw_s = (torch.zeros(K, C, dtype=torch.float64) for _ in range(3))
    db, db_e, db_s = (torch.zeros(C, dtype=torch.float64) for _ in range(3))
    for i, n in enumerate(lens):
        old = torch.zeros(K - 1, C, dtype=torch.float64) if s is None else s[i].double()
        ext, d = torch.cat([old, x[at:at + n].double()]), dy[at:at + n].double()
        z = sum(W[k] * ext[k:k + n] for k in range(K)) + B
        size = sum((W[k] * ext[k:k + n]).abs() for k in range(K)) + B.abs()
        if act == "silu":
            p, q = torch.sigmoid(z), torch.sigmoid(-z)
            e = d.abs() * (0.5 * (K + 1) * size + 2 * (z.abs() + 8) * (1 + z.abs())) * U
            d = d * p * (1 + z * q)
            e = e + U * d.abs()
        else:
            e = torch.zeros_like(d)
        dext, bound = torch.zeros_like(ext), torch.zeros_like(ext)
        for k in range(K):
            dext[k:k + n] += W[k] * d
            bound[k:k + n] += W[k].abs() * (e + K * U * d.abs())
            dw[k] += (d * ext[k:k + n]).sum(0)
            dw_e[k] += ((e * ext[k:k + n]) ** 2).sum(0)
            dw_s[k] += ((d * ext[k:k + n]) ** 2).sum(0)
        db += d.sum(0)
        db_e += (e ** 2).sum(0)
        db_s += (d ** 2).sum(0)
        if dso is not None:
            dext[n:] += dso[i].double()
            bound[n:] += K * U * dso[i].double().abs()
        bound += half * dext.abs()
        dxs.append((dext[K - 1:], bound[K - 1:]))
        dstates.append((dext[:K - 1], bound[:K - 1]))
        at += n
    joined = lambda parts, how: tuple(how([p[j] for p in parts]) for j in range(2))  # noqa: E731
    total = lambda v, e, t: (v, 4 * e.sqrt() + 2 * T ** 0.5 * U * t.sqrt() + U * v.abs())  # noqa: E731
    return [joined(dxs, torch.cat), total(dw, dw_e, dw_s), total(db, db_e, db_s),
            joined(dstates, torch.stack) if state else (None, None)]
