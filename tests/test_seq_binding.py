"""What the sequence operators' binding refuses before the library is called.
CPU only: no test here launches a kernel."""
import pytest
import torch

import depthwise_convolution_amd as dw
from depthwise_convolution_amd import seq

BIG = 2 ** 32 + 5  # a 32-bit int keeps 5 of it


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.fixture
def any_device(monkeypatch):
    """Tensors without memory stand in for the GPU's: what is checked comes
    before anything is allocated or launched."""
    monkeypatch.setattr(seq._Plan, "_device", lambda self, name, t: t.device)


def past_int(call, *args, **kwargs):
    with pytest.raises(ValueError, match="2147483647"):
        call(*args, **kwargs)


def test_counts_past_32_bits_are_refused_by_the_functions():
    h = dw.dwconv_causal_create(8, 4, "f32", "none")
    P = [1 << 20 | i << 12 for i in range(16)]
    past_int(dw.dwconv_causal_fwd, h, P[0], 8, P[1], None, P[2], BIG, 10, None, None, P[3], 8, None)
    past_int(dw.dwconv_causal_fwd, h, P[0], 8, P[1], None, P[2], 2, BIG, None, None, P[3], 8, None)
    past_int(dw.dwconv_causal_step, h, P[0], 8, P[1], None, P[2], P[3], BIG, 3, P[4], 8, None)
    past_int(dw.dwconv_causal_step, h, P[0], 8, P[1], None, P[2], P[3], 5, BIG, P[4], 8, None)
    past_int(dw.dwconv_causal_bwd_workspace, h, BIG)
    past_int(dw.dwconv_causal_bwd, h, P[0], 8, P[1], None, P[2], 2, BIG, None, P[3], 8, None, P[4], 8, P[5], None, None,
             P[6], None)
    dw.dwconv_causal_destroy(h)
    h = dw.dwconv_delta_create(1, 1, 8, 8, "f32", 1.0, True, 1e-6)
    past_int(dw.dwconv_delta_workspace, h, BIG, 10, False)
    past_int(dw.dwconv_delta_workspace, h, 1, BIG, True)
    past_int(dw.dwconv_delta_fwd, h, P[0], 8, P[1], 8, P[2], 8, P[3], P[4], P[5], 2, BIG, None, None, P[6], 8, P[7], None)
    past_int(dw.dwconv_delta_step, h, P[0], 8, P[1], 8, P[2], 8, P[3], P[4], P[5], P[6], 5, BIG, P[7], 8, None)
    past_int(dw.dwconv_delta_bwd, h, P[0], 8, P[1], 8, P[2], 8, P[3], P[4], P[5], BIG, 10, None, P[6], 8, None, P[7], 8,
             P[8], 8, P[9], 8, P[10], P[11], None, P[12], None)
    dw.dwconv_delta_destroy(h)
    p = dw.dwconv_norm_create(8, "f32", "none", "none", "none", 0.0)
    past_int(dw.dwconv_norm_fwd, p, BIG, P[0], None, None, 1, None, None, None, None, None, P[1], None, None)
    past_int(dw.dwconv_norm_fwd, p, 6, P[0], None, P[2], BIG, None, None, None, None, None, P[1], None, None)
    past_int(dw.dwconv_norm_bwd_workspace, p, BIG, 1)
    past_int(dw.dwconv_norm_bwd_workspace, p, 1, BIG)
    past_int(dw.dwconv_norm_bwd, p, BIG, P[0], *[None] * 2, 1, *[None] * 5, P[1], None, P[2], *[None] * 7, P[3], None)
    dw.dwconv_norm_destroy(p)


@pytest.mark.parametrize("call", [
    lambda: dw.dwconv_causal_create(BIG, 4, "f32", "none"), lambda: dw.dwconv_causal_create(8, 2 ** 32 + 4, "f32", "none"),
    lambda: dw.GatedDeltaRule(1, BIG, 8, 8), lambda: dw.GatedDeltaRule(1, 1, 2 ** 32 + 8, 8),
    lambda: dw.BlockNorm(BIG, "bf16"), lambda: dw.BlockNorm(8, "bf16", after=2 ** 32),
    lambda: dw.dwconv_delta_create(1, 1, 8, 8, 2 ** 32, 1.0, True, 1e-6),
])
def test_plans_past_32_bits_are_refused(call):
    past_int(call)


def test_counts_past_32_bits_are_refused_by_the_classes(any_device):
    x, w = meta(BIG, 8), meta(4, 8)
    conv = dw.CausalDepthwiseConv1d(8, 4, "f32")
    past_int(conv, x, w)
    past_int(conv, meta(5, 8), w, offsets=meta(BIG, dtype=torch.int32))
    past_int(conv.backward, x, w, x)
    past_int(conv.step, x, w, None, state=meta(BIG, 3, 8))
    past_int(conv.step, meta(5, 8), w, None, state=meta(BIG, 3, 8))
    rule = dw.GatedDeltaRule(1, 1, 8, 8, "f32")
    q, g = meta(BIG, 1, 8), meta(BIG, 1)
    past_int(rule, q, q, q, g, g)
    past_int(rule.backward, q, q, q, g, g, q)
    past_int(rule.step, q, q, q, g, g, state=meta(8, 1, 8, 8))
    past_int(rule.step, q[:5], q[:5], q[:5], g[:5], g[:5], state=meta(BIG, 1, 8, 8))
    norm = dw.BlockNorm(8, "f32")
    past_int(norm, x, w_after=meta(8), w_before=meta(8))
    past_int(norm.backward, x, x, x, w_after=meta(8), w_before=meta(8))
    past_int(norm, x[:6], gate=x[:1], rows_per_gate=BIG, w_after=meta(8), w_before=meta(8))


def test_grids_are_refused_before_anything_is_launched():
    """Where the last kernel's grid is the one that passes the limit, the call says
    so as it does for the others (here, without a GPU, a launch is another error)."""
    P = [1 << 20 | i << 16 for i in range(16)]

    def unsupported(call, *args):
        with pytest.raises(dw.DwconvError) as e:
            call(*args)
        assert e.value.status == 2

    # one unit of 65536 heads x 62 groups of columns, rounded up to eight units
    h = dw.dwconv_delta_create(1, 65536, 8, 1984, "bf16", 1.0, True, 1e-6)
    wide = 65536 * 1984
    unsupported(dw.dwconv_delta_fwd, h, P[0], 8, P[1], 8, P[2], wide, P[3], P[4], None, 1, 64, None, None, P[5], wide,
                P[6], None)
    unsupported(dw.dwconv_delta_bwd, h, P[0], 8, P[1], 8, P[2], wide, P[3], P[4], None, 1, 64, None, P[5], wide, None,
                P[6], 8, P[7], 8, P[8], wide, P[9], P[10], None, P[11], None)
    dw.dwconv_delta_destroy(h)
    # the sums of 5 x 2^29 columns
    h = dw.dwconv_causal_create(1 << 29, 4, "bf16", "none")
    unsupported(dw.dwconv_causal_bwd, h, P[0], 1 << 29, P[1], None, None, 1, 1, None, P[2], 1 << 29, None, P[3], 1 << 29,
                P[4], None, None, P[5], None)
    dw.dwconv_causal_destroy(h)
    # a step's groups of columns count as its rows and heads do
    h = dw.dwconv_delta_create(1, 64, 8, 4096, "bf16", 1.0, True, 1e-6)
    unsupported(dw.dwconv_delta_step, h, P[0], 8, P[1], 8, P[2], 64 * 4096, P[3], P[4], P[5], P[6], 5, 1 << 13, P[7],
                64 * 4096, None)
    dw.dwconv_delta_destroy(h)


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="cuda:1"):
        seq._on(torch.device("cuda", 0), Stream(), lambda raw: pytest.fail("called"))


def test_a_tensor_that_requires_a_gradient_is_refused(any_device):
    """Before anything is allocated or launched, on every entry point."""
    def r(*shape):
        return meta(*shape).requires_grad_()

    x, w, q, v, g, one = meta(6, 8), meta(4, 8), meta(6, 1, 8), meta(6, 2, 8), meta(6, 2), meta(8)
    conv, rule, norm = dw.CausalDepthwiseConv1d(8, 4, "f32"), dw.GatedDeltaRule(1, 2, 8, 8, "f32"), dw.BlockNorm(8, "f32")
    for call in (lambda: conv(x, r(4, 8)), lambda: conv.step(x, w, r(8), state=meta(6, 3, 8)),
                 lambda: conv.backward(x, w, r(6, 8)), lambda: rule(q, q, v, r(6, 2), g),
                 lambda: rule.step(q, q, v, g, g, state=r(6, 2, 8, 8)), lambda: rule.backward(q, q, v, g, g, r(6, 2, 8)),
                 lambda: norm(x, r(6, 8), w_after=one, w_before=one),
                 lambda: norm.backward(x, x, x, gate=r(6, 8), w_after=one, w_before=one)):
        with pytest.raises(ValueError, match="autograd"):
            call()


def test_counts_near_2_to_the_31_are_refused():
    """Kernels add a run, a chunk or one to a count of tokens or sequences."""
    h = dw.dwconv_causal_create(8, 4, "bf16", "silu")
    r = dw.dwconv_delta_create(1, 1, 8, 8, "bf16", 1.0, True, 1e-6)
    P = [1 << 20 | i << 16 for i in range(16)]
    most = 2 ** 31 - 129
    for n in (most + 1, 2 ** 31 - 1):
        for call in (lambda: dw.dwconv_causal_fwd(h, P[0], 8, P[1], None, P[2], n, 10, None, None, P[3], 8, None),
                     lambda: dw.dwconv_causal_fwd(h, P[0], 8, P[1], None, P[2], 2, n, None, None, P[3], 8, None),
                     lambda: dw.dwconv_causal_bwd(h, P[0], 8, P[1], None, P[2], n, 10, None, P[3], 8, None, P[4], 8, P[5],
                                                  None, None, P[6], None),
                     lambda: dw.dwconv_causal_bwd_workspace(h, n), lambda: dw.dwconv_delta_workspace(r, n, 10, False),
                     lambda: dw.dwconv_delta_workspace(r, 1, n, True),
                     lambda: dw.dwconv_delta_fwd(r, P[0], 8, P[1], 8, P[2], 8, P[3], P[4], P[5], n, 10, None, None, P[6],
                                                 8, P[7], None)):
            with pytest.raises(dw.DwconvError) as e:
                call()
            assert e.value.status == 1
    assert dw.dwconv_causal_bwd_workspace(h, most) > dw.dwconv_causal_bwd_workspace(h, most - 2 ** 20)
    # as many sequences as the delta rule's grid does not hold are told apart from bad ones
    with pytest.raises(dw.DwconvError) as e:
        dw.dwconv_delta_fwd(r, P[0], 8, P[1], 8, P[2], 8, P[3], P[4], P[5], most, most, None, None, P[6], 8, P[7], None)
    assert e.value.status == 2
    dw.dwconv_causal_destroy(h)
    dw.dwconv_delta_destroy(r)
