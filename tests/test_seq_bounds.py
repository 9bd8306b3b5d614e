"""The bounds of the sequence operators' GPU tests see what they are meant to
see: a mistake planted in the 64-bit form fails them, fp32 arithmetic passes.
CPU only."""
import math

import pytest
import torch

import seq_reference as ref
from seq_cases import CONV_GRADS, conv_grad_bounds, conv_grad_data, in_terms, readback, readback_bound


@pytest.mark.parametrize("Dk", [16, 64, 128, 192, 256])
def test_readback_bound_sees_two_terms(Dk):
    """One chunk in its chunked form: the state, P and U in two bf16 terms
    (2^-18) are outside the bound of the read-back, three terms and plain fp32
    sums well inside."""
    q, k, v, _, _, state = readback("bf16", 1, 1, Dk, 48, [64])
    k = k[:, 0].double()
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    v, S, scale = v[:, 0].double(), state[0, 0].double(), Dk ** -0.5

    def chunk(terms, dt=torch.float64):
        K, V, S0 = k.to(dt), v.to(dt), S.to(dt)
        T = torch.linalg.inv(torch.eye(64, dtype=torch.float64) + (k @ k.T).tril(-1)).to(dt)
        u = T @ (V - K @ S0)
        P = scale * (K @ K.T).tril()
        if terms:
            S0, P, u = in_terms(S0, terms), in_terms(P, terms), in_terms(u, terms)
        return (scale * (K @ S0) + P @ u).double()

    exact, c = chunk(0), scale * (k @ S)
    bound = readback_bound(torch.bfloat16, exact, c, Dk)
    off = lambda x: float((x - exact).norm())  # noqa: E731
    assert off(chunk(2)) > 1.2 * bound
    assert off(chunk(3)) < 0.3 * bound and off(chunk(0, torch.float32)) < 0.6 * bound
    assert math.isfinite(bound)


@pytest.mark.parametrize("case", CONV_GRADS, ids=lambda c: f"{c[0]}-C{c[1]}-K{c[2]}-{sum(c[3])}-{c[4]}")
def test_conv_gradient_bounds(case):
    """They are those of the definition; gradients kept in 16 bits, or summed in
    them, are outside; sums in fp32 are inside."""
    fmt, C, K, lens, act, state = case
    x, w, b, s, dy, dso = conv_grad_data(case)
    (dx, dx_b), (dw_, dw_b), (db, db_b), (ds, ds_b) = conv_grad_bounds(case, x, w, b, s, dy, dso)
    xs, ws, bs, ss = ref.leaves(x, w, b, s)
    y, st, _, _ = ref.conv(xs, ws, bs, lens, ss, act)
    outs, gives, wrt = ([y, st], [dy.double(), dso.double()], [xs, ws, bs, ss]) if state else ([y], [dy.double()], [xs, ws, bs])
    for a, g in zip(torch.autograd.grad(outs, wrt, gives), (dx, dw_, db, ds)):
        assert torch.allclose(a, g, rtol=1e-11, atol=1e-11)

    def outside(got, want, bound):
        off = (got.double() - want).abs()
        return bool((off > bound).any()) or float(off.norm()) > 0.5 * float(bound.norm())

    for v, bound in ((dw_, dw_b), (db, db_b)):
        assert outside(v.to(torch.bfloat16), v, bound) and outside(v.to(torch.float16), v, bound)
        assert not outside(v.float(), v, bound)
    assert not outside(dx.to(x.dtype), dx, dx_b)
    if fmt == "f32":
        assert outside(dx.to(torch.float16), dx, dx_b) and outside(dx.to(torch.bfloat16), dx, dx_b)
    if fmt == "f16":
        assert outside(dx.to(torch.bfloat16), dx, dx_b)
    # bias gradients added one by one in 16 bits and in 32
    if act == "none" and len(lens) < 3:
        for dt, bad in ((torch.bfloat16, True), (torch.float32, False)):
            run = torch.zeros(4, dtype=dt)
            for row in dy[:, :4].double():
                run = (run.double() + row).to(dt)
            assert outside(run, db[:4], db_b[:4]) == bad
