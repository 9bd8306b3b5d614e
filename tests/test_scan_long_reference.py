"""The long form of the scan's 64-bit reference is the short one's, and its cases take the runs
that they are meant to take.  CPU only."""
import pytest
import torch

import depthwise_convolution_amd as dw
import scan_reference as ref
from scan_cases import scan_data
from scan_long import LONG, linear, long_bounds, long_id
from seq_reference import DTYPES

NAMES = ("x", "dt", "a", "b", "c", "skip", "bias", "gate")


@pytest.mark.parametrize("T", [1, 2, 7, 100, 101])
def test_linear_recurrence(T):
    g = torch.Generator().manual_seed(T)
    e, put, h = torch.rand(T, 3, generator=g).double(), torch.randn(T, 3, generator=g).double(), torch.ones(3).double()
    got = linear(e, put, h)
    for t in range(T):
        h = e[t] * h + put[t]
        assert torch.allclose(got[t], h, rtol=1e-13, atol=1e-13)


@pytest.mark.parametrize("case", [("f32", 6, 5, 2, [130], True, "silu", True, True, 0), ("bf16", 3, 4, 1, [77], True, "sigmoid", True, True, 0),
                                  ("f16", 4, 2, 4, [50], False, None, False, False, 0), ("f32", 2, 3, 1, [1], True, "silu", True, True, 0)],
                         ids=str)
def test_long_form_is_the_short_one(case):
    fmt, C, N, G, lens, state, act, soft, _, _ = case
    d = scan_data(case, seed=5)
    args = [d[n] for n in NAMES]
    st = None if d["state"] is None else d["state"][0]
    dst = None if d["dstate"] is None else d["dstate"][0]
    want = ref.scan_bounds(DTYPES[fmt], *args, lens, d["state"], soft, act, d["dy"], d["dstate"])
    got = long_bounds(DTYPES[fmt], *args, st, soft, act, d["dy"], dst)
    for k, (value, bound) in got.items():
        assert torch.allclose(value, want[k][0], rtol=1e-10, atol=1e-12), k
        assert torch.allclose(bound, want[k][1], rtol=1e-6, atol=1e-18), k


@pytest.mark.parametrize("case", LONG, ids=long_id)
def test_cases_run_in_the_runs_they_stand_for(case):
    """Read off the forward workspace: 1024 states and 256 / lanes widths a run, and as many
    places for runs as tokens / length + sequences."""
    fmt, C, N, G, lens, _, run = case
    lanes = 4 if N <= 16 else 8 if N <= 32 else 16 if N <= 64 else 32
    assert C * lanes <= 256, "more than one block of channels"
    h = dw.dwconv_scan_create(C, N, G, fmt, True, "silu")
    need = dw.dwconv_scan_workspace(h, len(lens), sum(lens), False)
    assert need == 4 * (sum(lens) // run + len(lens)) * (1024 + 256 // lanes)
    back = dw.dwconv_scan_workspace(h, len(lens), sum(lens), True)
    runs, kept = sum(lens) // run + len(lens), sum(lens) // 8 + len(lens)
    walkers = min(runs, 2048)
    assert back == 4 * (runs * (2048 + 256 // lanes) + kept * 1024 + sum(lens) * 8 * lanes + walkers * (1024 + 512 // lanes))
    dw.dwconv_scan_destroy(h)
