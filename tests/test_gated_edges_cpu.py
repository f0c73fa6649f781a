"""More refusals of the gated block's operators, and what their workspaces hold."""
import ctypes

import pytest

from state_space_model_scan_amd import _lib
from tests.test_gated_cpu import FAKE, _norm_bwd


def _wide(rows, cols, group, **kw):
    return _norm_bwd(rows=rows, cols=cols, group_size=group,
                     **{k + "_stride": cols for k in ("x", "z", "dy", "ds", "dx", "dresidual", "dz")}, **kw)


def _size(a):
    size = ctypes.c_size_t()
    assert _lib.lib().rms_norm_bwd_workspace_size(ctypes.byref(a), ctypes.byref(size)) == _lib.SSM_OK
    return size.value


def test_norm_bwd_refuses_a_workspace_off_4_bytes():
    """... and one that is missing or too small, before anything is launched."""
    L, need = _lib.lib(), _size(_wide(3000, 256, 128))
    assert need > 0
    for kw, want in ((dict(), _lib.SSM_ERR_WORKSPACE), (dict(workspace=FAKE, workspace_bytes=need - 1), _lib.SSM_ERR_WORKSPACE),
                     (dict(workspace=FAKE + 2, workspace_bytes=need), _lib.SSM_ERR_UNSUPPORTED),
                     (dict(workspace=FAKE + 1, workspace_bytes=need), _lib.SSM_ERR_UNSUPPORTED)):
        assert L.rms_norm_bwd(ctypes.byref(_wide(3000, 256, 128, **kw)), None) == want, kw


@pytest.mark.parametrize("rows,cols,group", [(1 << 20, 2560, 2560), (1 << 20, 4096, 8), (200001, 512, 1), (131072, 5120, 80),
                                             ((1 << 31) - 1, 2, 1)])
def test_norm_bwd_workspace_of_many_rows(rows, cols, group):
    """A workgroup's sums are of at most 256 rows a lane: a unit is at least 8
    lanes of at most 256 threads (512 of the largest groups)."""
    blocks = _size(_wide(rows, cols, group)) // (4 * cols)
    assert blocks * 32 * 256 >= rows
