"""The bounds of the sequence operators' GPU tests see what they are meant to
see: a mistake planted in the 64-bit form fails them, fp32 arithmetic passes.
CPU only."""
import math

import pytest
import torch

from seq_cases import in_terms, readback, readback_bound


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
