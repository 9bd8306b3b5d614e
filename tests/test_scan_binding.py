"""What the selective scan and the group norm refuse before anything is launched,
through the C ABI's functions and the classes.  CPU only."""
import pytest
import torch

import depthwise_convolution_amd as dw
from depthwise_convolution_amd import seq

BIG = 2 ** 32 + 5
P = [(1 << 30) + (i << 16) for i in range(32)]  # addresses that are never read


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.fixture
def any_device(monkeypatch):
    """Tensors without memory stand in for the GPU's: what is checked comes
    before anything is allocated or launched."""
    monkeypatch.setattr(seq._Plan, "_device", lambda self, name, t: t.device)


def status_of(call, *args):
    with pytest.raises(dw.DwconvError) as e:
        call(*args)
    return e.value.status


@pytest.mark.parametrize("args", [
    (0, 16, 1, "f32"), (8, 0, 1, "f32"), (8, 129, 1, "f32"), (8, 16, 0, "f32"), (8, 16, 3, "f32"), (-8, 16, 1, "f32"),
    (2 ** 24 + 1, 1, 1, "f32"), (8, 16, 16, "f32"), (8, 16, 1, "i8"),
])
def test_scan_plans_refused(args):
    assert status_of(dw.dwconv_scan_create, *args, True, "silu") == 1


def test_plans_with_unknown_choices():
    with pytest.raises(ValueError):
        dw.SelectiveScan(8, 16, gate_act="relu")
    with pytest.raises(ValueError):
        dw.GroupNorm(8, 2, act="sigmoid")
    assert status_of(dw.dwconv_scan_create, 8, 16, 1, "f32", True, 3) == 1
    assert status_of(dw.dwconv_group_create, 8, 2, "f32", 3, 1e-5) == 1
    assert status_of(dw.dwconv_group_create, 8, 2, "f32", -1, 1e-5) == 1


@pytest.mark.parametrize("args", [
    (0, 1, "f32", "silu", 1e-5), (8, 0, "f32", "silu", 1e-5), (8, 3, "f32", "silu", 1e-5), (8, 16, "f32", "silu", 1e-5),
    (65537, 1, "f32", "silu", 1e-5), (8, 2, "i8", "silu", 1e-5), (8, 2, "f32", "silu", -1e-5),
    (8, 2, "f32", "silu", float("nan")), (8, 2, "f32", "silu", float("inf")),
])
def test_group_plans_refused(args):
    assert status_of(dw.dwconv_group_create, *args) == 1


def scan_args(**change):
    a = dict(x=P[0], ldx=8, dt=P[1], lddt=8, a=P[2], b=P[3], ldb=4, c=P[4], ldc=4, skip=P[5], dt_bias=P[6], gate=P[7],
             ldgate=8)
    rest = {k: change.pop(k) for k in list(change) if k not in a}
    a.update(change)
    return list(a.values()), rest


def call_scan(kind, h, **change):
    args, rest = scan_args(**change)
    g = lambda k, v: rest.get(k, v)  # noqa: E731
    if kind == "fwd":
        return dw.dwconv_scan_fwd(h, *args, g("offsets", P[8]), g("seqs", 2), g("n", 5), g("state_in", P[9]),
                                  g("state_out", P[10]), g("y", P[11]), g("ldy", 8), g("ws", P[12]), None)
    if kind == "step":
        return dw.dwconv_scan_step(h, *args, g("state", P[9]), g("slots", P[8]), g("n_slots", 6), g("n", 5), g("y", P[11]),
                                   g("ldy", 8), None)
    return dw.dwconv_scan_bwd(h, *args, g("offsets", P[8]), g("seqs", 2), g("n", 5), g("state_in", P[9]), g("dy", P[13]),
                              g("lddy", 8), g("dstate_out", P[10]), g("dx", P[14]), g("lddx", 8), g("ddt", P[15]),
                              g("ldddt", 8), g("da", P[16]), g("db", P[17]), g("lddb", 4), g("dc", P[18]), g("lddc", 4),
                              g("dskip", P[19]), g("ddt_bias", P[20]), g("dgate", P[21]), g("lddgate", 8),
                              g("dstate_in", P[22]), g("ws", P[12]), None)


COMMON = [dict(x=None), dict(dt=None), dict(a=None), dict(b=None), dict(c=None), dict(ldx=7), dict(lddt=7), dict(ldb=3),
          dict(ldc=3), dict(ldgate=7), dict(x=P[0] + 1), dict(a=P[2] + 2), dict(skip=P[5] + 2), dict(gate=P[7] + 1),
          dict(dt_bias=P[6] + 1), dict(n=-1), dict(ldx=2 ** 62)]
SEQS = [dict(offsets=None), dict(offsets=P[8] + 2), dict(seqs=-1), dict(seqs=2 ** 31 - 1), dict(n=2 ** 31 - 1),
        dict(state_in=P[9] + 2), dict(ws=P[12] + 4)]
KINDS = {
    "fwd": COMMON + SEQS + [dict(y=None), dict(y=P[0]), dict(y=P[1]), dict(y=P[7]), dict(y=P[11] + 1), dict(ldy=7),
                            dict(state_out=P[9] + 4), dict(state_out=P[10] + 1)],
    "step": COMMON + [dict(y=None), dict(y=P[0]), dict(y=P[7]), dict(ldy=7), dict(state=None), dict(state=P[9] + 2),
                      dict(n_slots=-1), dict(slots=None, n=7), dict(slots=P[8] + 1)],
    "bwd": COMMON + SEQS + [dict(dy=None), dict(dx=None), dict(ddt=None), dict(da=None), dict(db=None), dict(dc=None),
                            dict(ws=None), dict(dx=P[0]), dict(dx=P[13]), dict(ddt=P[1]), dict(dgate=P[7]), dict(db=P[3]),
                            dict(da=P[2]), dict(lddx=7), dict(ldddt=7), dict(lddb=3), dict(lddc=3), dict(lddgate=7),
                            dict(dstate_in=P[9]), dict(dstate_in=P[10] + 4), dict(da=P[16] + 1), dict(dskip=P[19] + 2)],
}


@pytest.mark.parametrize("kind,change", [(k, c) for k, cs in KINDS.items() for c in cs], ids=str)
def test_scan_calls_refused(kind, change):
    h = dw.dwconv_scan_create(8, 4, 1, "f32", True, "silu")
    assert status_of(lambda: call_scan(kind, h, **change)) == 1
    assert status_of(lambda: call_scan(kind, None, **change)) == 1
    dw.dwconv_scan_destroy(h)


def call_group(back, h, **change):
    a = dict(images=2, pixels=3, x=P[0], ldx=8, w=P[1], b=P[2], dy=P[3], lddy=8, y=P[4], ldy=8, dw=P[5], db=P[6], ws=P[7])
    a.update(change)
    head = [h, a["images"], a["pixels"], a["x"], a["ldx"], a["w"], a["b"]]
    if back:
        return dw.dwconv_group_bwd(*head, a["dy"], a["lddy"], a["y"], a["ldy"], a["dw"], a["db"], a["ws"], None)
    return dw.dwconv_group_fwd(*head, a["y"], a["ldy"], a["ws"], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("change", [
    dict(images=-1), dict(pixels=-1), dict(images=2 ** 16, pixels=2 ** 15), dict(x=None), dict(y=None), dict(ldx=7), dict(ldy=7),
    dict(x=P[0] + 2), dict(w=P[1] + 1), dict(b=P[2] + 2), dict(y=P[4] + 1), dict(ws=P[7] + 8), dict(ldx=2 ** 62),
], ids=str)
def test_group_calls_refused(back, change):
    h = dw.dwconv_group_create(8, 2, "f32", "silu", 1e-5)
    assert status_of(lambda: call_group(back, h, **change)) == 1
    assert status_of(lambda: call_group(back, None)) == 1
    dw.dwconv_group_destroy(h)


@pytest.mark.parametrize("back,change", [
    (False, dict(y=P[0], ldy=9)), (True, dict(dy=None)), (True, dict(y=P[0])), (True, dict(y=P[3], ldy=9)), (True, dict(ws=None)),
    (True, dict(lddy=7)), (True, dict(dw=P[5] + 2)), (True, dict(db=P[6] + 1)), (True, dict(dy=P[3] + 2)),
], ids=str)
def test_group_calls_refused_one_way(back, change):
    h = dw.dwconv_group_create(8, 2, "f32", "silu", 1e-5)
    assert status_of(lambda: call_group(back, h, **change)) == 1
    dw.dwconv_group_destroy(h)


def test_a_missing_workspace_is_refused_where_one_is_needed():
    h = dw.dwconv_scan_create(64, 16, 1, "f32", True, "silu")
    assert dw.dwconv_scan_workspace(h, 1, 60, False) == 0 and dw.dwconv_scan_workspace(h, 1, 100000, False) > 0
    assert dw.dwconv_scan_workspace(h, 1, 60, True) > 0
    args, _ = scan_args(ldx=64, lddt=64, ldb=16, ldc=16, ldgate=64)
    assert status_of(lambda: dw.dwconv_scan_fwd(h, *args, None, 1, 100000, None, None, P[11], 64, None, None)) == 1
    dw.dwconv_scan_destroy(h)
    h = dw.dwconv_group_create(64, 4, "f32", "silu", 1e-5)
    assert dw.dwconv_group_workspace(h, 2, 10 ** 6, False) > 0
    assert status_of(lambda: dw.dwconv_group_fwd(h, 2, 10 ** 6, P[0], 64, None, None, P[1], 64, None, None)) == 1
    dw.dwconv_group_destroy(h)


def test_workspaces_hold_what_a_call_keeps():
    """A state of every 16 tokens, whatever the lengths; more tokens never need less."""
    for C, N, G in ((8192, 16, 1), (33, 5, 1), (64, 100, 4)):
        h = dw.dwconv_scan_create(C, N, G, "bf16", True, "silu")
        last = 0
        for n in (0, 1, 16, 1000, 4096, 100000):
            need = dw.dwconv_scan_workspace(h, 3, n, True)
            assert need >= 4 * (n // 16) * C * N and need >= last
            last = need
        dw.dwconv_scan_destroy(h)


def test_grids_that_pass_their_limit_are_unsupported():
    h = dw.dwconv_scan_create(2 ** 24, 1, 1, "f32", True, "none")
    wide = dict(ldx=2 ** 24, lddt=2 ** 24, ldgate=2 ** 24, ldb=1, ldc=1)
    assert status_of(lambda: call_scan("fwd", h, seqs=64, n=64, ldy=2 ** 24, state_in=None, state_out=None, **wide)) == 2
    assert status_of(lambda: call_scan("step", h, n=64, ldy=2 ** 24, n_slots=64, **wide)) == 2
    assert status_of(lambda: call_scan("bwd", h, seqs=64, n=64, lddy=2 ** 24, lddx=2 ** 24, ldddt=2 ** 24, lddb=1, lddc=1,
                                       lddgate=2 ** 24, state_in=None, dstate_out=None, dstate_in=None, **wide)) == 2
    assert dw.dwconv_scan_workspace(h, 64, 64, True) == 2 ** 64 - 1
    dw.dwconv_scan_destroy(h)
    h = dw.dwconv_scan_create(8, 4, 1, "f32", True, "silu")
    for name in ("ldx", "lddt", "ldb", "ldc", "ldgate", "ldy"):
        assert status_of(lambda: call_scan("fwd", h, **{name: 2 ** 26 + 1})) == 2
    for name in ("ldx", "lddt", "ldb", "ldc", "ldgate", "lddy", "lddx", "ldddt", "lddb", "lddc", "lddgate"):
        assert status_of(lambda: call_scan("bwd", h, **{name: 2 ** 26 + 1})) == 2
    dw.dwconv_scan_destroy(h)
    h = dw.dwconv_group_create(65536, 65536, "f32", "none", 1e-5)
    assert status_of(lambda: call_group(False, h, images=2 ** 20, pixels=1, ldx=65536, ldy=65536)) == 2
    assert status_of(lambda: call_group(True, h, images=2 ** 20, pixels=1, ldx=65536, ldy=65536, lddy=65536)) == 2
    dw.dwconv_group_destroy(h)


def past(call):
    with pytest.raises(ValueError, match="2147483647"):
        call()


def test_counts_past_32_bits_are_refused(any_device):
    past(lambda: dw.SelectiveScan(BIG, 16))
    past(lambda: dw.SelectiveScan(8, 2 ** 32 + 16))
    past(lambda: dw.GroupNorm(BIG, 1))
    h = dw.dwconv_scan_create(8, 4, 1, "f32", True, "silu")
    for kind, names in (("fwd", ("seqs", "n")), ("step", ("n_slots", "n")), ("bwd", ("seqs", "n"))):
        for name in names:
            past(lambda: call_scan(kind, h, **{name: BIG}))
    past(lambda: dw.dwconv_scan_workspace(h, BIG, 3, False))
    past(lambda: dw.dwconv_scan_workspace(h, 3, BIG, True))
    dw.dwconv_scan_destroy(h)
    h = dw.dwconv_group_create(8, 2, "f32", "silu", 1e-5)
    for name in ("images", "pixels"):
        past(lambda: call_group(False, h, **{name: BIG}))
        past(lambda: call_group(True, h, **{name: BIG}))
    past(lambda: dw.dwconv_group_workspace(h, BIG, 1, False))
    dw.dwconv_group_destroy(h)
    scan, x, a, b = dw.SelectiveScan(8, 4, 1, "f32"), meta(BIG, 8), meta(8, 4), meta(BIG, 1, 4)
    past(lambda: scan(x, x, a, b, b))
    past(lambda: scan.backward(x, x, a, b, b, x))
    past(lambda: scan.step(x, x, a, b, b, meta(6, 8, 4)))
    past(lambda: scan.step(x[:5], x[:5], a, b[:5], b[:5], meta(BIG, 8, 4)))
    group = dw.GroupNorm(8, 2, "f32")
    past(lambda: group(meta(BIG, 3, 8)))
    past(lambda: group(meta(2 ** 20, 2 ** 12, 8)))


def test_classes_check_shapes_types_and_strides(any_device):
    scan = dw.SelectiveScan(8, 4, 2, "f32")
    x, a, b = meta(6, 8), meta(8, 4), meta(6, 2, 4)
    good = dict(x=x, dt=x, a=a, b=b, c=b)
    bad = [dict(x=meta(6, 9)), dict(x=meta(6, 8, dtype=torch.float16)), dict(x=meta(6, 16)[:, ::2]), dict(dt=meta(5, 8)),
           dict(a=meta(4, 8).t()), dict(a=meta(8, 4, dtype=torch.float16)), dict(b=meta(6, 1, 4)), dict(c=meta(6, 2, 8)[:, :, ::2]),
           dict(b=meta(6, 2, 8)[:, :, :4]), dict(skip=meta(9)), dict(dt_bias=meta(8, 1)), dict(gate=meta(7, 8)),
           dict(gate=meta(8, 6).t())]
    for change in bad:
        k = {**good, **change}
        pos = [k.pop(n) for n in ("x", "dt", "a", "b", "c")]
        for call in (lambda: scan(*pos, **k), lambda: scan.step(*pos, meta(6, 8, 4), **k), lambda: scan.backward(*pos, x, **k)):
            with pytest.raises(ValueError):
                call()
    pos = [x, x, a, b, b]
    for call in (lambda: scan(*pos, state_in=meta(2, 8, 4)), lambda: scan(*pos, state_out=meta(1, 4, 8)),
                 lambda: scan(*pos, offsets=meta(3)), lambda: scan.step(*pos, meta(5, 8, 4)),
                 lambda: scan.step(*pos, meta(6, 4, 8)), lambda: scan.step(*pos, meta(9, 8, 4), slots=meta(6)),
                 lambda: scan.backward(*pos, meta(6, 9)), lambda: scan.backward(*pos, x, dstate_out=meta(2, 8, 4)),
                 lambda: scan(x[0], x, a, b, b)):
        with pytest.raises(ValueError):
            call()
    group = dw.GroupNorm(8, 2, "f32")
    x = meta(2, 5, 3, 8)
    for call in (lambda: group(meta(2, 5, 3, 9)), lambda: group(meta(8)), lambda: group(x.transpose(1, 2)),
                 lambda: group(meta(2, 5, 6, 8)[:, :, :3]), lambda: group(meta(2, 5, 3, 16)[..., ::2]),
                 lambda: group(x, meta(9)), lambda: group(x, None, meta(8, dtype=torch.float16)),
                 lambda: group(meta(2, 5, 3, 8, dtype=torch.float16)), lambda: group.backward(x, meta(2, 15, 8))):
        with pytest.raises(ValueError):
            call()


def test_closed_plans_tensors_on_the_host_and_gradients_are_refused(any_device, monkeypatch):
    scan, group = dw.SelectiveScan(8, 4, 1, "f32"), dw.GroupNorm(8, 2, "f32")
    x, a, b = meta(6, 8), meta(8, 4), meta(6, 1, 4)
    r = lambda *s: meta(*s).requires_grad_()  # noqa: E731
    for call in (lambda: scan(r(6, 8), x, a, b, b), lambda: scan(x, x, r(8, 4), b, b), lambda: scan.step(x, x, a, b, b, r(6, 8, 4)),
                 lambda: scan.backward(x, x, a, b, b, r(6, 8)), lambda: scan(x, x, a, b, b, gate=r(6, 8)),
                 lambda: group(r(2, 3, 8)), lambda: group(meta(2, 3, 8), r(8)), lambda: group.backward(meta(2, 3, 8), r(2, 3, 8))):
        with pytest.raises(ValueError, match="autograd"):
            call()
    monkeypatch.undo()
    cpu = torch.zeros(6, 8)
    with pytest.raises(ValueError, match="GPU"):
        scan(cpu, cpu, torch.zeros(8, 4), torch.zeros(6, 1, 4), torch.zeros(6, 1, 4))
    with pytest.raises(ValueError, match="GPU"):
        group(torch.zeros(2, 3, 8))
    scan.close()
    group.close()
    scan.close()
    with pytest.raises(ValueError, match="closed"):
        scan(cpu, cpu, cpu, cpu, cpu)
    with pytest.raises(ValueError, match="closed"):
        group(cpu)
