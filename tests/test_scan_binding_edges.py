"""What the selective scan and the group norm refuse, and the workspaces they ask for, where
tests/test_scan_binding.py does not reach.  CPU only: no test here launches a kernel."""
import pytest

import depthwise_convolution_amd as dw

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
