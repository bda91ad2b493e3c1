"""Outputs and inputs of the scan's gradient that are columns of one tensor: refused where they
share an element, not where they lie side by side. No GPU: what lies side by side is shown by the
check that comes after (two outputs that coincide), so that nothing is ever launched."""
import ctypes

import pytest

from mamba_selective_scan_sm_b200 import _abi
from tests.test_abi_bwd_host import FAKE, bwd, lib  # noqa: F401

ES, D, N = 2, 64, 16
U, DU, DDELTA, B = FAKE, FAKE + (6 << 28), FAKE + (7 << 28), FAKE + (3 << 28)


def answer(lib, **kw):  # noqa: F811
    a = bwd(channel_last=1, dC=FAKE + (9 << 28), dB=FAKE + (9 << 28), **kw)   # dB and dC coincide
    status = _abi.STATUS[lib.ssm_selective_scan_bwd(ctypes.byref(a), None)]
    return status, lib.ssm_last_error_detail().decode()


@pytest.mark.parametrize("kw", [
    dict(stride_u=4 * D, stride_du=4 * D, du=U + 2 * D * ES),             # u | z | du | dz
    dict(stride_u=4 * D, stride_du=4 * D, du=U + D * ES),                 # right behind u
    dict(stride_u=4 * D, stride_du=4 * D, u=DU + D * ES, du=DU),          # before it
    dict(stride_u=4 * D, stride_du=4 * D, du=U + 3 * D * ES),             # the last columns
    dict(stride_B=D + N, stride_du=D + N, du=B + N * ES),                 # of different widths
])
def test_side_by_side(lib, kw):  # noqa: F811
    assert answer(lib, **kw) == ("SSM_ERR_ALIAS", "dC overlaps dB")


@pytest.mark.parametrize("kw,names", [
    (dict(stride_u=4 * D, stride_du=4 * D, du=U + (D - 1) * ES), "du overlaps u"),       # one element
    (dict(stride_u=4 * D, stride_du=4 * D, du=U + (3 * D + 1) * ES), "du overlaps u"),   # into the next row
    (dict(stride_u=4 * D, stride_du=3 * D, du=U + 2 * D * ES), "du overlaps u"),         # other steps
    (dict(stride_u=2 * D, du=U + D * ES), "du overlaps u"),                              # dense beside strided
    (dict(stride_B=D + N, stride_du=D + N, du=B + (N - 1) * ES), "du overlaps B"),
])
def test_shared_elements(lib, kw, names):  # noqa: F811
    assert answer(lib, **kw) == ("SSM_ERR_ALIAS", names)
