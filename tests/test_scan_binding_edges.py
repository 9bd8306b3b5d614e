"""What the selective scan and the group norm refuse, and the workspaces they ask for, where
tests/test_scan_binding.py does not reach.  CPU only: no test here launches a kernel."""
import pytest
import torch

import depthwise_convolution_amd as dw
from depthwise_convolution_amd import seq

P = [(1 << 40) + (i << 16) for i in range(16)]  # addresses that are never read


def status_of(call, *args):
    with pytest.raises(dw.DwconvError) as e:
        call(*args)
    return e.value.status


@pytest.mark.parametrize("back, pixels, images", [(False, 4000, 2048), (True, 2000, 4096)])
def test_group_grids_of_wide_workgroups_are_unsupported(back, pixels, images):
    """Images that workgroups of 1024 lanes (512 in the gradients) hold in registers, 2048
    workgroups each: 2^32 lanes."""
    h = dw.dwconv_group_create(65536, 4096, "bf16", "none", 1e-5)
    if back:
        assert dw.dwconv_group_workspace(h, images, pixels, True) == images * 2 * 65536 * 4, "not in registers"
        assert status_of(dw.dwconv_group_bwd, h, images, pixels, P[0], 65536, None, None, P[1], 65536, P[2], 65536, None, None,
                         P[3], None) == 2
    else:
        assert dw.dwconv_group_workspace(h, images, pixels, False) == 0, "not in registers"
        assert status_of(dw.dwconv_group_fwd, h, images, pixels, P[0], 65536, None, None, P[1], 65536, None, None) == 2
    dw.dwconv_group_destroy(h)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_scans_without_a_workspace_that_memory_could_hold_are_unsupported(monkeypatch, back, given):
    """The library gives the workspace's size of a grid past its limit as SIZE_MAX, which is
    no size to allocate.  (64 tokens of 2^24 channels; no memory stands behind the tensors.)"""
    monkeypatch.setattr(seq._Plan, "_device", lambda self, name, t: t.device)
    monkeypatch.setattr(seq, "_on", lambda dev, stream, body, *tensors: body(0))
    meta = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    C = 2 ** 24
    plan, x, b = dw.SelectiveScan(C, 1, 1, "f32"), meta(64, C), meta(64, 1, 1)
    named = dict(offsets=meta(65, dtype=torch.int32), workspace=meta(1 << 20, dtype=torch.uint8) if given else None)
    if back:
        assert status_of(lambda: plan.backward(x, x, meta(C, 1), b, b, x, **named)) == 2
    else:
        assert status_of(lambda: plan(x, x, meta(C, 1), b, b, **named)) == 2


def test_scan_workspaces_hold_a_state_of_every_8_tokens():
    for C, N, G in ((8192, 16, 1), (33, 5, 1), (64, 100, 4), (96, 24, 3)):
        h = dw.dwconv_scan_create(C, N, G, "bf16", True, "silu")
        for seqs in (1, 3):
            for n in (0, 1, 8, 1000, 4096, 100000):
                assert dw.dwconv_scan_workspace(h, seqs, n, True) >= 4 * (n // 8 + seqs) * C * N
        dw.dwconv_scan_destroy(h)
