"""The 64-bit forms of the sequence operators against differences, against
each other and against closed cases; argument checks of the C ABI and of the
binding.  CPU only: no test here launches a kernel."""
import ctypes
import math

import pytest
import torch

import depthwise_convolution_amd as dw
import seq_reference as ref

PTR = 1 << 20  # an aligned non-null pointer that nothing dereferences


def gen(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed + 17 * len(shape) + sum(shape))
    return torch.randn(shape, generator=g, dtype=torch.float64) * std


def test_conv_is_torch_conv1d():
    x, w, b = gen(20, 6), gen(4, 6, seed=1), gen(6, seed=2)
    y, state, _, _ = ref.conv(x, w, b, [20], None, "none")
    lib = torch.nn.functional.conv1d(torch.nn.functional.pad(x.t()[None], (3, 0)), w.t()[:, None], b, groups=6)
    assert torch.allclose(y, lib[0].t(), atol=1e-13)
    assert torch.equal(state[0], x[-3:])


def test_conv_continues_from_its_state():
    x, w = gen(11, 5), gen(3, 5, seed=1)
    whole, last, _, _ = ref.conv(x, w, None, [11], None, "silu")
    first, mid, _, _ = ref.conv(x[:1], w, None, [1], None, "silu")
    rest, end, _, _ = ref.conv(x[1:], w, None, [10], mid, "silu")
    assert torch.equal(torch.cat([first, rest]), whole) and torch.equal(end, last)


def test_delta_closed_cases():
    n, H, D = 5, 2, 3
    q, k, v = gen(n, H, D), gen(n, H, D, seed=1), gen(n, H, 4, seed=2)
    zero, one = torch.zeros(n, H, dtype=torch.float64), torch.ones(n, H, dtype=torch.float64)
    # beta = 0 keeps the state; no decay
    S0 = gen(1, H, D, 4, seed=3)
    o, S, _ = ref.delta(q, k, v, zero, zero, [n], S0, 1.0, False, 0.0)
    assert torch.equal(S, S0) and torch.allclose(o, (S0[0] * q[..., None]).sum(2))
    # beta = 1 with a unit key stores the value under it exactly
    o, S, _ = ref.delta(q, k, v, zero, one, [n], S0, 1.0, True, 0.0)
    unit = k[-1] / k[-1].norm(dim=-1, keepdim=True)
    assert torch.allclose((S[0] * unit[..., None]).sum(1), v[-1])
    # g = -inf forgets: every token sees itself alone
    o, S, _ = ref.delta(q, k, v, torch.full_like(zero, -math.inf), one, [n], S0, 1.0, False, 0.0)
    assert torch.allclose(o, (q * k).sum(-1, keepdim=True) * v)


def test_gradients_match_differences():
    n = 4
    q, k, v = gen(n, 1, 3), gen(n, 1, 3, seed=1), gen(n, 2, 2, seed=2)
    g, b, S = -gen(n, 2, seed=3).abs(), torch.sigmoid(gen(n, 2, seed=4)), gen(2, 2, 3, 2, seed=5)
    args = [t.requires_grad_() for t in (q, k, v, g, b, S)]
    assert torch.autograd.gradcheck(lambda *a: ref.delta(*a[:5], [3, 1], a[5], 0.5, True, 1e-6)[:2], args)
    args = [t.requires_grad_() for t in (gen(5, 3), gen(3, 3, seed=1), gen(3, seed=2), gen(2, 2, 3, seed=3))]
    assert torch.autograd.gradcheck(lambda x, w, c, s: ref.conv(x, w, c, [4, 1], s, "silu")[:2], args)
    for after, before in (("rms", "layer"), ("layer", "rms")):
        args = [t.requires_grad_() for t in (gen(4, 5), gen(4, 5, seed=1), gen(2, 5, seed=2)) +
                tuple(gen(5, seed=3 + i) for i in range(5))]
        assert torch.autograd.gradcheck(
            lambda o, r, gt, s, wa, ba, wb, bb: ref.block(o, r, gt, 2, s, wa, ba, wb, bb, after, before, "silu", 1e-6),
            args)


# --- refusals ----------------------------------------------------------------
@pytest.mark.parametrize("args", [
    (0, 4, "bf16", "silu"), (8, 1, "bf16", "silu"), (8, 9, "f32", "none"), (8, 4, "i8", "none"), (8, 4, 7, "none"),
    (8, 4, "f16", "sigmoid"), (8, 4, "f16", 5), (-3, 4, "f16", "none"),
])
def test_causal_create_refuses(args):
    with pytest.raises(dw.DwconvError) as e:
        dw.dwconv_causal_create(*args)
    assert e.value.status == 1


@pytest.mark.parametrize("args", [
    (0, 1, 8, 8, "bf16", 1.0, 1, 1e-6), (2, 3, 8, 8, "bf16", 1.0, 1, 1e-6), (1, 1, 0, 8, "bf16", 1.0, 1, 1e-6),
    (1, 1, 257, 8, "bf16", 1.0, 1, 1e-6), (1, 1, 8, 0, "bf16", 1.0, 1, 1e-6), (1, 1, 8, 4097, "f32", 1.0, 1, 1e-6),
    (1, 1, 8, 8, "i8", 1.0, 1, 1e-6), (1, 1, 8, 8, "f32", math.nan, 1, 1e-6), (1, 1, 8, 8, "f32", 1.0, 1, -1.0),
    (1, 1, 8, 8, "f32", math.inf, 1, 0.0),
])
def test_delta_create_refuses(args):
    with pytest.raises(dw.DwconvError) as e:
        dw.dwconv_delta_create(*args)
    assert e.value.status == 1


@pytest.mark.parametrize("args", [
    (0, "bf16", "rms", "rms", "silu", 1e-6), (16385, "bf16", "rms", "rms", "silu", 1e-6),
    (8, "i8", "rms", "rms", "silu", 1e-6), (8, "f32", 3, "rms", "silu", 1e-6), (8, "f32", "rms", -1, "silu", 1e-6),
    (8, "f32", "rms", "rms", 3, 1e-6), (8, "f32", "rms", "rms", "silu", math.nan),
])
def test_norm_create_refuses(args):
    with pytest.raises(dw.DwconvError) as e:
        dw.dwconv_norm_create(*args)
    assert e.value.status == 1


def test_unknown_choices():
    with pytest.raises(ValueError):
        dw.CausalDepthwiseConv1d(8, 4, "bf16", act="gelu")
    with pytest.raises(ValueError):
        dw.BlockNorm(8, "bf16", after="batch")
    with pytest.raises(ValueError):
        dw.GatedDeltaRule(1, 1, 8, 8, "f64")


def refused(call, *args):
    with pytest.raises(dw.DwconvError) as e:
        call(*args)
    assert e.value.status == 1


def vary(call, good, changes):
    """Each change to the good arguments is refused before any launch."""
    for i, v in changes:
        args = list(good)
        args[i] = v
        refused(call, *args)


def test_causal_arguments():
    h = dw.dwconv_causal_create(8, 4, "bf16", "silu")
    P = [PTR + (i << 12) for i in range(16)]
    try:
        # h x ldx w bias offsets seqs tokens state_in state_out y ldy stream
        fwd = (h, P[0], 8, P[1], P[2], P[3], 2, 10, P[4], P[5], P[6], 8, None)
        vary(dw.dwconv_causal_fwd, fwd, [
            (0, None), (1, None), (1, P[0] + 1), (2, 7), (3, None), (3, P[1] + 1), (4, P[2] + 2), (5, None),
            (5, P[3] + 2), (6, -1), (7, -1), (7, 2 ** 31 - 1), (9, P[4]), (9, P[4] + 16), (8, P[4] + 1), (10, None),
            (10, P[0]), (11, 0), (11, -8)])
        # h x ldx w bias state slots n_slots rows y ldy stream
        step = (h, P[0], 8, P[1], P[2], P[3], P[4], 5, 3, P[5], 8, None)
        vary(dw.dwconv_causal_step, step, [
            (0, None), (1, None), (3, None), (5, None), (5, P[3] + 1), (6, P[4] + 1), (7, -1), (8, -1), (9, None),
            (9, P[0]), (10, 4)])
        refused(dw.dwconv_causal_step, h, P[0], 8, P[1], None, P[3], None, 2, 3, P[5], 8, None)  # rows > entries
        bwd = (h, P[0], 8, P[1], P[2], P[3], 2, 10, P[4], P[5], 8, P[6], P[7], 8, P[8], P[9], P[10], P[11], None)
        vary(dw.dwconv_causal_bwd, bwd, [
            (0, None), (1, None), (3, None), (5, None), (9, None), (10, 7), (12, None), (12, P[0]), (12, P[5]),
            (13, 7), (14, None), (14, P[8] + 2), (16, P[6]), (16, P[4] + 32), (17, None), (17, P[11] + 2)])
        refused(dw.dwconv_causal_bwd_workspace, h, -1)
        refused(dw.dwconv_causal_bwd_workspace, None, 1)
        assert dw.dwconv_causal_bwd_workspace(h, 0) == 0
        assert dw.dwconv_causal_bwd_workspace(h, 1) >= 5 * 8 * 4
    finally:
        dw.dwconv_causal_destroy(h)
    dw.dwconv_causal_destroy(None)


def test_delta_arguments():
    h = dw.dwconv_delta_create(2, 4, 8, 16, "f16", 1.0, True, 1e-6)
    P = [PTR + (i << 16) for i in range(24)]
    try:
        # h q ldq k ldk v ldv g beta offsets seqs tokens state_in state_out o ldo ws stream
        fwd = (h, P[0], 16, P[1], 16, P[2], 64, P[3], P[4], P[5], 2, 10, P[6], P[7], P[8], 64, P[9], None)
        vary(dw.dwconv_delta_fwd, fwd, [
            (0, None), (1, None), (2, 15), (3, P[1] + 1), (4, -16), (5, None), (6, 63), (7, None), (8, P[4] + 1),
            (9, None), (10, -1), (11, -1), (13, P[6] + 64), (14, None), (14, P[2]), (15, 63), (16, None),
            (16, P[9] + 4)])
        # h q ldq k ldk v ldv g beta state slots n_slots rows o ldo stream
        step = (h, P[0], 16, P[1], 16, P[2], 64, P[3], P[4], P[5], P[6], 5, 3, P[7], 64, None)
        vary(dw.dwconv_delta_step, step, [
            (0, None), (1, None), (6, 8), (7, None), (9, None), (9, P[5] + 2), (10, P[6] + 1), (11, -2), (12, -1),
            (13, None), (13, P[0])])
        refused(dw.dwconv_delta_step, h, P[0], 16, P[1], 16, P[2], 64, P[3], P[4], P[5], None, 2, 3, P[7], 64, None)
        bwd = (h, P[0], 16, P[1], 16, P[2], 64, P[3], P[4], P[5], 2, 10, P[6], P[7], 64, P[8], P[9], 16, P[10], 16,
               P[11], 64, P[12], P[13], P[14], P[15], None)
        vary(dw.dwconv_delta_bwd, bwd, [
            (0, None), (1, None), (9, None), (13, None), (14, 1), (16, None), (16, P[0]), (17, 15), (18, P[13 - 11]),
            (20, None), (20, P[7]), (21, 63), (22, None), (22, P[3]), (23, None), (24, P[6]), (24, P[8] + 64),
            (25, None), (25, P[15] + 8)])
        for bad in ((-1, 1), (1, -1)):
            refused(dw.dwconv_delta_workspace, h, *bad, False)
        f, b = (dw.dwconv_delta_workspace(h, 3, 1000, x) for x in (False, True))
        assert 0 < f < b
    finally:
        dw.dwconv_delta_destroy(h)
    dw.dwconv_delta_destroy(None)


def test_norm_arguments():
    p = dw.dwconv_norm_create(8, "bf16", "rms", "layer", "silu", 1e-6)
    P = [PTR + (i << 12) for i in range(32)]
    try:
        # p rows o res gate per scale wa ba wb bb h y stream
        fwd = (p, 6, P[0], P[1], P[2], 2, P[3], P[4], None, P[5], P[6], P[7], P[8], None)
        vary(dw.dwconv_norm_fwd, fwd, [
            (0, None), (1, -1), (2, None), (2, P[0] + 1), (5, 0), (6, P[3] + 2), (7, None), (9, None), (12, None),
            (12, P[7]), (12, P[1]), (11, P[0] + 16), (11, P[1] + 16)])
        bwd = (p, 6, P[0], P[1], P[2], 2, P[3], P[4], None, P[5], P[6], P[7], P[8], P[9], P[10], P[11], P[12], P[13],
               None, P[14], P[15], P[16], None)
        vary(dw.dwconv_norm_bwd, bwd, [
            (0, None), (1, -1), (2, None), (5, 0), (7, None), (9, None), (12, None), (13, P[0]), (13, P[7]),
            (14, P[8]), (14, P[9]), (15, P[2]), (15, P[0] + 16), (16, P[12] + 2), (21, None), (21, P[16] + 1)])
        refused(dw.dwconv_norm_bwd_workspace, p, -1, 1)
        refused(dw.dwconv_norm_bwd_workspace, p, 1, 0)
    finally:
        dw.dwconv_norm_destroy(p)
    q = dw.dwconv_norm_create(8, "bf16", "none", "none", "none", 0.0)
    try:
        refused(dw.dwconv_norm_fwd, q, 6, P[0], None, None, 1, None, None, None, None, None, None, P[8], None)  # no h
    finally:
        dw.dwconv_norm_destroy(q)
    dw.dwconv_norm_destroy(None)


def test_null_results_of_create():
    lib = ctypes.CDLL(dw.library_path)
    assert lib.dwconv_causal_create(None, 8, 4, 0, 0) == 1
    lib.dwconv_delta_create.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 5 + [ctypes.c_float, ctypes.c_int,
                                                                                 ctypes.c_float]
    assert lib.dwconv_delta_create(None, 1, 1, 8, 8, 0, 1.0, 1, 0.0) == 1
    lib.dwconv_norm_create.argtypes = [ctypes.c_void_p] + [ctypes.c_int] * 5 + [ctypes.c_float]
    assert lib.dwconv_norm_create(None, 8, 0, 1, 1, 1, 0.0) == 1


def test_host_tensors_are_refused():
    x, w = torch.zeros(4, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError):
        dw.CausalDepthwiseConv1d(8, 4, "f32")(x, w)
    with pytest.raises(ValueError):
        dw.BlockNorm(8, "f32")(x)
    with pytest.raises(ValueError):
        dw.GatedDeltaRule(1, 1, 8, 8, "f32")(x, x, x, x, x)


def test_workspaces_cover_every_partition():
    """The norm's partial sums: what the deal of rows to workgroups needs never
    exceeds what the query says (rows x group sizes around its thresholds)."""
    for D in (1, 96, 128, 129, 512, 2048, 2049, 16384):
        p = dw.dwconv_norm_create(D, "f32", "layer", "layer", "silu", 1e-6)
        try:
            for rows in (0, 1, 15, 16, 17, 1000, 2048, 2049, 200704):
                for per in (1, 2, 7, 3136, rows + 1):
                    n = dw.dwconv_norm_bwd_workspace(p, rows, per)
                    assert n % (4 * D) == 0 and (n > 0) == (rows > 0)
        finally:
            dw.dwconv_norm_destroy(p)


def test_grids_past_their_limit_are_unsupported():
    """Refused before anything is launched, whatever the pointers."""
    P = [PTR + (i << 16) for i in range(12)]

    def unsupported(call, *args):
        with pytest.raises(dw.DwconvError) as e:
            call(*args)
        assert e.value.status == 2

    h = dw.dwconv_causal_create(8, 4, "bf16", "silu")
    unsupported(dw.dwconv_causal_step, h, P[0], 8, P[1], None, P[2], P[3], 5, 1 << 24, P[4], 8, None)
    dw.dwconv_causal_destroy(h)
    h = dw.dwconv_delta_create(1, 64, 8, 8, "bf16", 1.0, True, 1e-6)
    unsupported(dw.dwconv_delta_step, h, P[0], 8, P[1], 8, P[2], 512, P[3], P[4], P[5], P[6], 5, 1 << 18, P[7], 512,
                None)
    unsupported(dw.dwconv_delta_fwd, h, P[0], 8, P[1], 8, P[2], 512, P[3], P[4], P[5], 1 << 16, 64, None, None, P[6],
                512, P[7], None)
    dw.dwconv_delta_destroy(h)
