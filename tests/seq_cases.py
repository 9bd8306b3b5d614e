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
