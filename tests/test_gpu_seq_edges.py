"""The sequence operators on the GPU where they are easily wrong: sums that
cancel, values that are not numbers, borders.  Bounds are derived in
tests/seq_cases.py and shown on planted mistakes in tests/test_seq_bounds.py."""
import pytest
import torch

import depthwise_convolution_amd as dw
import seq_reference as ref
from gpu_helpers import DEV, say
from seq_cases import readback, readback_bound, readback_terms
from test_gpu_seq import offsets_of, up

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
