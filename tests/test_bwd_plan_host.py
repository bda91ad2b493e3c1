"""The workspace that the scan's gradient asks for, on the host (no GPU): what it depends on, and
that a batch which fills the GPU is not cut into segments."""
import ctypes

import pytest

from mamba_selective_scan_sm_b200 import _abi
from tests.test_abi_bwd_host import P, bwd, lib  # noqa: F401


def size(lib, **kw):  # noqa: F811
    n = ctypes.c_size_t()
    assert lib.ssm_selective_scan_bwd_workspace_size(ctypes.byref(bwd(workspace=None, **kw)), ctypes.byref(n)) == 0
    return n.value


SHAPES = [dict(batch=8, dim=1536, seqlen=2048), dict(batch=1, dim=5120, seqlen=16384), dict(batch=1, dim=64, seqlen=256),
          dict(batch=1, dim=1, seqlen=1), dict(batch=3, dim=100, seqlen=1 << 20), dict(batch=60000, dim=1, seqlen=3)]


@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("dstate,heads", [(1, 0), (4, 1), (8, 0), (16, 0), (16, 1), (24, 0), (64, 0), (128, 0), (128, 1)])
def test_neither_packing_nor_strides_change_it(lib, kw, dtype, dstate, heads):  # noqa: F811
    """A caller may keep one workspace for calls from values and from 8-bit codes, with or without
    z, states and optional gradients."""
    kw = dict(kw, dtype=dtype, dstate=dstate, a_heads=heads)
    for cl in (0, 1):
        plain = size(lib, channel_last=cl, **kw)
        assert plain == size(lib, channel_last=cl, u_scale=P, delta_scale=P, **kw)
        assert plain == size(lib, channel_last=cl, z=P, dz=P, initial_state=P, dfinal_state=P, dD=P, **kw)
        assert plain == size(lib, channel_last=cl, stride_u=1 << 20, stride_du=1 << 21, **{**kw, "dim": kw["dim"]})


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("dstate,heads", [(4, 0), (16, 0), (16, 8), (128, 0), (128, 8)])
def test_many_rows_are_one_segment(lib, dtype, dstate, heads):  # noqa: F811
    kw = dict(batch=64, dim=4096, seqlen=64, dtype=dtype, dstate=dstate, a_heads=heads)
    assert size(lib, **kw) == size(lib, num_segments=1, **kw)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("dstate", [4, 16, 128])
def test_one_narrow_row_is_cut(lib, dtype, dstate):  # noqa: F811
    kw = dict(batch=1, dim=64, seqlen=65536, dtype=dtype, dstate=dstate)
    assert size(lib, **kw) > size(lib, num_segments=1, **kw)
