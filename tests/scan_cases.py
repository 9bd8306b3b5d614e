"""Inputs that the CPU and the GPU tests of the selective scan and the group
norm share."""
import torch

from seq_reference import DTYPES

# fmt, C, N, G, lengths, state, gate activation (None: no gate), softplus, skip and bias, channels more a token
SCAN = [
    ("bf16", 64, 16, 1, [1], False, "silu", True, True, 0),
    ("f32", 70, 16, 1, [16, 17, 1], True, "silu", True, True, 0),
    ("f16", 61, 11, 1, [5, 0, 2, 33], True, "sigmoid", True, True, 3),
    ("bf16", 130, 16, 2, [200, 3], True, "silu", True, True, 6),
    ("f32", 7, 1, 7, [0, 0, 90], False, "none", True, False, 0),
    ("bf16", 96, 24, 3, [33, 31, 2, 1, 70], True, None, True, True, 32),
    ("f16", 40, 64, 2, [130], False, "silu", True, True, 5),
    ("f32", 33, 50, 1, [64, 65], True, None, False, True, 0),
    ("bf16", 20, 128, 1, [100, 7], True, "silu", True, True, 0),
    ("f32", 12, 100, 4, [70, 90], True, "sigmoid", True, False, 1),
    ("bf16", 1, 5, 1, [40, 6], True, "silu", True, True, 0),
    ("f32", 100, 16, 1, [1500], True, "silu", True, True, 0),
    ("f16", 256, 16, 1, [700, 1, 2, 300], True, "silu", True, True, 0),
    ("bf16", 8, 16, 1, [1, 2, 0, 3, 1] * 500, True, "silu", True, True, 0),
    ("f32", 1024, 100, 1, [150] * 7, True, "silu", True, True, 0),
]


def scan_id(c):
    return f"{c[0]}-C{c[1]}-N{c[2]}-G{c[3]}-{len(c[4])}x{sum(c[4])}-{c[6]}"


def scan_data(case, seed=0, grad=True):
    """x, dt, a, b, c, skip, bias, gate, state, dy, dstate on the CPU."""
    fmt, C, N, G, lens, state, act, soft, params, _ = case
    g = torch.Generator().manual_seed(1000 * seed + C + 7 * N + 31 * sum(lens) + len(lens))
    T, dt = sum(lens), DTYPES[fmt]
    r = lambda *s, std=1.0: torch.randn(*s, generator=g) * std  # noqa: E731
    width = r(T, C, std=1.0).to(dt) if soft else (torch.rand(T, C, generator=g) * 0.5).to(dt)
    a = -torch.exp(r(C, N, std=0.3)) * torch.arange(1, N + 1) * (16 / N if N > 16 else 1.0)
    bias = None
    if params:
        bias = r(C, std=1.0) - 3 if soft else torch.rand(C, generator=g) * 0.1
    return dict(x=r(T, C).to(dt), dt=width, a=a, b=r(T, G, N).to(dt), c=r(T, G, N).to(dt),
                skip=r(C) if params else None, bias=bias, gate=None if act is None else r(T, C).to(dt),
                state=r(len(lens), C, N, std=0.5) if state else None, dy=r(T, C).to(dt) if grad else None,
                dstate=r(len(lens), C, N, std=0.3) if state and grad else None)


# fmt, images, pixels, C, G, activation, weights, channels more a pixel
GROUP = [
    ("bf16", 1, 64, 512, 32, "silu", True, 0),
    ("f32", 2, 49, 128, 32, "silu", True, 0),
    ("f16", 3, 100, 96, 32, "silu", True, 0),
    ("bf16", 2, 169, 61, 61, "none", True, 0),
    ("f32", 1, 1, 6, 2, "silu", True, 0),
    ("bf16", 2, 1, 1, 1, "none", True, 0),
    ("f16", 2, 7, 5, 1, "relu", True, 0),
    ("f32", 2, 33, 3, 3, "silu", False, 2),
    ("bf16", 2, 300, 40, 4, "silu", True, 24),
    ("f16", 2, 50, 50, 10, "relu", True, 3),
    ("f32", 1, 5000, 8, 2, "silu", True, 0),
    ("bf16", 1, 3, 4096, 1, "silu", True, 0),
    ("f32", 1, 70, 2051, 1, "silu", True, 0),
    ("bf16", 2, 20, 6200, 2, "none", True, 0),
    ("f16", 1, 9, 2500, 2500, "none", False, 0),
    ("f32", 40, 4, 16, 4, "silu", True, 0),
    ("bf16", 1, 3136, 64, 16, "silu", True, 0),
    ("f16", 1, 13000, 24, 8, "silu", True, 0),
    ("f32", 1, 40000, 4, 1, "silu", True, 0),
    ("bf16", 3, 784, 33, 11, "silu", True, 1),
    ("bf16", 1, 5000, 32, 2, "silu", True, 0),
    ("f16", 2, 2900, 64, 4, "silu", True, 0),
    ("bf16", 1, 600000, 8, 1, "none", True, 0),
    ("f32", 1, 9000, 256, 2, "silu", True, 0),
    ("f32", 1, 9000, 256, 2, "none", True, 0),
    ("f16", 16, 2500, 61, 61, "none", True, 0),
    ("f32", 1, 36000, 256, 8, "none", True, 0),
    ("f32", 1, 720000, 3, 1, "none", True, 0),
]


def group_id(c):
    return f"{c[0]}-{c[1]}x{c[2]}-C{c[3]}-G{c[4]}-{c[5]}"


def group_data(case, seed=0):
    """x, w, b, dy on the CPU; means of some deviations."""
    fmt, n, S, C, G, act, params, _ = case
    g = torch.Generator().manual_seed(1000 * seed + C + 7 * S + 31 * n)
    dt = DTYPES[fmt]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(n, S, C) * (0.5 + torch.rand(C, generator=g)) + 3 * r(G).repeat_interleave(C // G)).to(dt)
    w, b = (0.5 + torch.rand(C, generator=g), r(C) * 0.3) if params else (None, None)
    return dict(x=x, w=w, b=b, dy=r(n, S, C).to(dt))
