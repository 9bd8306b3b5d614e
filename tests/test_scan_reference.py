"""The 64-bit forms of the selective scan and the group norm: their gradients
against autograd's and against differences, their bounds against fp32 arithmetic
(inside) and planted mistakes (outside).  CPU only."""
import pytest
import torch

import scan_reference as ref
from scan_cases import GROUP, SCAN, group_data, group_id, scan_data, scan_id
from seq_reference import DTYPES, leaves, starts

SMALL = [c for c in SCAN if sum(c[4]) * c[1] * c[2] < 4e6]
NAMES = ("x", "dt", "a", "b", "c", "skip", "bias", "gate")


@pytest.mark.parametrize("case", SMALL, ids=scan_id)
def test_scan_recurrences_are_autograds(case):
    fmt, C, N, G, lens, state, act, soft, _, _ = case
    d = scan_data(case)
    got = ref.scan_bounds(DTYPES[fmt], *(d[n] for n in NAMES), lens, d["state"], soft, act, d["dy"], d["dstate"])
    ls = dict(zip(NAMES + ("state",), leaves(*(d[n] for n in NAMES + ("state",)))))
    y, st = ref.scan(*(ls[n] for n in NAMES), lens, ls["state"], soft, act)
    assert torch.allclose(y, got["y"][0], rtol=1e-11, atol=1e-11) and torch.allclose(st, got["state"][0], rtol=1e-11, atol=1e-11)
    outs, gives = [y], [d["dy"].double()]
    if state:
        outs, gives = outs + [st], gives + [d["dstate"].double()]
    wrt = {n: t for n, t in ls.items() if t is not None}
    for (n, _), v in zip(wrt.items(), torch.autograd.grad(outs, list(wrt.values()), gives)):
        assert torch.allclose(v, got["d" + n][0], rtol=1e-10, atol=1e-10), n


def test_scan_gradients_are_differences():
    case = ("f32", 4, 3, 2, [3, 2], True, "silu", True, True, 0)
    d = scan_data(case)
    ls = leaves(*(d[n] for n in NAMES), d["state"])
    assert torch.autograd.gradcheck(lambda *t: ref.scan(*t[:8], case[4], t[8]), ls)


@pytest.mark.parametrize("case", [c for c in SMALL if sum(c[4]) > 8], ids=scan_id)
def test_scan_bounds_see_16_bits(case):
    """States kept in 16 bits between tokens, or decays rounded to them, are outside;
    the definition in fp32 is inside."""
    fmt, C, N, G, lens, state, act, soft, _, _ = case
    d = scan_data(case)
    want = ref.scan_bounds(DTYPES[fmt], *(d[n] for n in NAMES), lens, d["state"], soft, act)
    y, st = ref.scan(*(None if d[n] is None else d[n].float() for n in NAMES), lens, d["state"], soft, act)
    assert not ref.outside(y.to(DTYPES[fmt]), *want["y"]) and not ref.outside(st, *want["state"])
    assert ref.outside(st.to(torch.float16), *want["state"]) and ref.outside(st.to(torch.bfloat16), *want["state"])
    if fmt == "f32":
        assert ref.outside(y.to(torch.float16), *want["y"])
    a = d["a"].to(torch.float16).float()  # rates
    bad = ref.scan(d["x"].double(), d["dt"].double(), a.double(), *(None if d[n] is None else d[n].double() for n in NAMES[3:]),
                   lens, None if d["state"] is None else d["state"].double(), soft, act)[1]
    assert ref.outside(bad, *want["state"])
    # a state carried from one sequence into the next
    if len(lens) > 1 and all(lens) and not state:
        bad = ref.scan(*(None if d[n] is None else d[n].double() for n in NAMES), [sum(lens)], None, soft, act)[0]
        assert ref.outside(bad, *want["y"])
    assert starts(lens)[-1] == sum(lens)


@pytest.mark.parametrize("case", GROUP, ids=group_id)
def test_group_recurrences_are_autograds_and_bounds_hold_fp32(case):
    fmt, n, S, C, G, act, _, _ = case
    d = group_data(case)
    got = ref.group_bounds(DTYPES[fmt], d["x"], d["w"], d["b"], G, act, 1e-5, d["dy"])
    ls = leaves(d["x"], d["w"], d["b"])
    y = ref.group(*ls, G, act, 1e-5)
    assert torch.allclose(y, got["y"][0], rtol=1e-10, atol=1e-10)
    wrt = [t for t in ls if t is not None]
    for k, v in zip(("dx", "dw", "db"), torch.autograd.grad(y, wrt, d["dy"].double())):
        assert torch.allclose(v, got[k][0], rtol=1e-8, atol=1e-8), k
    assert act != "relu" or got["border"] > 1, "a value of z within its error of the corner"
    plain = ref.group(d["x"].float(), d["w"], d["b"], G, act, 1e-5)
    assert not ref.outside(plain.to(DTYPES[fmt]), *got["y"])
    if S * C // G > 8 and fmt == "f32":  # a mean that is off by what sums in fp16 leave
        v = d["x"].double().view(n, S, G, C // G)
        v = v - v.mean((1, 3), keepdim=True) - 2.0 ** -11 * v.abs().mean((1, 3), keepdim=True)
        u = (v / torch.sqrt((v * v).mean((1, 3), keepdim=True) + 1e-5)).view(n, S, C)
        z = u if d["w"] is None else u * d["w"].double() + d["b"].double()
        assert ref.outside(ref.act_of(z, act), *got["y"])


def test_group_gradients_are_differences():
    d = group_data(("f32", 2, 3, 6, 2, "silu", True, 0))
    ls = leaves(d["x"], d["w"], d["b"])
    assert torch.autograd.gradcheck(lambda x, w, b: ref.group(x, w, b, 2, "silu", 1e-5), ls)
