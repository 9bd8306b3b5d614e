"""The sequence operators on the GPU where they are easily wrong: sums that
cancel, values that are not numbers, borders.  Bounds are derived in
tests/seq_cases.py and shown on planted mistakes in tests/test_seq_bounds.py."""
import pytest
import torch

import depthwise_convolution_amd as dw
import seq_reference as ref
from gpu_helpers import DEV, say
from seq_cases import readback, readback_bound, readback_terms
from test_gpu_seq import delta_data, offsets_of, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,Hk,Hv,Dk,Dv,lens", [
    ("bf16", 1, 2, 128, 48, [64, 70, 3]), ("f16", 1, 2, 128, 48, [64, 70, 3]), ("f32", 1, 2, 128, 48, [64, 70, 3]),
    ("bf16", 2, 2, 64, 33, [130]), ("f16", 1, 1, 64, 64, [1, 65]), ("bf16", 1, 1, 192, 40, [100]),
    ("f16", 1, 1, 192, 40, [100]), ("bf16", 1, 1, 256, 40, [100]), ("f16", 1, 1, 256, 32, [70]),
    ("bf16", 1, 3, 128, 70, [66, 64, 1] * 20), ("f16", 1, 3, 100, 70, [66, 64, 1] * 20),
], ids=str)
def test_delta_reads_back_what_it_stored(fmt, Hk, Hv, Dk, Dv, lens):
    """Outputs that are a small difference of large terms keep fp32 accuracy of
    the terms, whatever type o is rounded to."""
    say(f"[gpu] delta read-back {fmt} {Hk} {Hv} {Dk} {Dv} {lens[:4]}")
    q, k, v, g, beta, state = readback(fmt, Hk, Hv, Dk, Dv, lens)
    scale = Dk ** -0.5
    o = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, fmt)(*(up(t) for t in (q, k, v, g, beta)), offsets=offsets_of(lens),
                                               state_in=up(state))
    want, _, _ = ref.delta(*(t.double() for t in (q, k, v, g, beta)), lens, state.double(), scale, True, 1e-6)
    c = readback_terms(q, k, lens, state, v, scale, 1e-6)
    off, bound = float((o.double().cpu() - want).norm()), readback_bound(v.dtype, want, c, Dk)
    print(f"{fmt} Dk={Dk}: off {off / bound:.2f} of the bound", flush=True)
    assert off <= bound


# ---------------------------------------------------------------------------
# values that are not numbers
# ---------------------------------------------------------------------------
NAN, INF = float("nan"), float("inf")
SPOIL = [("v", NAN), ("v", INF), ("v", -INF), ("k", NAN), ("k", INF), ("q", NAN), ("beta", NAN), ("g", NAN),
         ("state", NAN), ("beta", INF)]


def of_head(name, h, group):
    """The value heads that head h of tensor `name` belongs to."""
    return list(range(h * group, (h + 1) * group)) if name in ("q", "k") else [h]


@pytest.mark.parametrize("name,bad", SPOIL, ids=lambda x: str(x))
@pytest.mark.parametrize("fmt,Hk,Hv,Dk,Dv,lens,chunk_first", [
    ("f32", 1, 2, 40, 70, [130, 70], 64), ("bf16", 1, 2, 128, 70, [130, 70], 64), ("f16", 2, 4, 64, 40, [130, 70], 64),
    ("bf16", 1, 3, 100, 70, [130, 70] * 16, 64), ("f16", 1, 1, 250, 33, [130, 70], 0), ("bf16", 1, 5, 72, 24, [90, 70], 64),
], ids=lambda x: str(x)[:12])
def test_delta_forward_is_causal_for_what_is_no_number(fmt, Hk, Hv, Dk, Dv, lens, chunk_first, name, bad):
    """A NaN or infinity at token t: the outputs of the tokens before it, of other
    sequences, other heads and (for v and the state) other columns keep their
    bits; its own and the later ones of its column are no numbers either."""
    say(f"[gpu] delta spoiled {fmt} {Hk} {Hv} {Dk} {Dv} {name} {bad}")
    data = [t for t in delta_data(fmt, Hk, Hv, Dk, Dv, lens, True, gates="plain", seed=7)]
    names = ["q", "k", "v", "g", "beta", "state"]
    rule, off, group = dw.GatedDeltaRule(Hk, Hv, Dk, Dv, fmt), offsets_of(lens), Hv // Hk

    def run(t):
        end = torch.empty_like(t[5])
        return rule(*t[:5], offsets=off, state_in=t[5], state_out=end), end

    clean, clean_end = run([up(t) for t in data])
    assert torch.isfinite(clean).all()
    # first and last token of a chunk, inside a tile of 16, in the second chunk
    for t in {chunk_first, chunk_first + 1, chunk_first + 21, min(chunk_first + 63, lens[0] - 1)}:
        d = [x.clone() for x in data]
        h = 1 if d[names.index(name)].shape[1] > 1 else 0
        col = Dv - 1
        if name == "state":
            d[5][0, h, 3, col] = bad
            t = 0
        elif name in ("g", "beta"):
            d[names.index(name)][t, h] = bad
        else:
            d[names.index(name)][t, h, col if name == "v" else 3] = bad
        o, end = run([up(x) for x in d])
        hit = torch.zeros_like(o, dtype=torch.bool)
        heads = of_head(name, h, group)
        cols = slice(col, col + 1) if name in ("v", "state") else slice(0, Dv)
        hit[t:t + 1 if name == "q" else lens[0], heads, cols] = True
        assert torch.equal(o[~hit], clean[~hit]), (t, "an output that must not see it changed")
        assert not torch.isfinite(o[hit]).any(), (t, "an output that must show it is a number")
        ends = torch.zeros_like(end, dtype=torch.bool)
        if name != "q":
            ends[0, heads, :, cols] = True
        assert torch.equal(end[~ends], clean_end[~ends]) and not torch.isfinite(end[ends]).any()
