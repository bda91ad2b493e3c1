"""Host-side checks of the training and cache entry points (no GPU): struct mirrors, workspace
sizes, and refusals before anything is launched. Pointers are fake and never dereferenced."""
import ctypes
import os
import subprocess

import pytest

from mamba_selective_scan_sm_b200 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from mamba_selective_scan_sm_b200 import build
        build.build()
    return _abi.load()


@pytest.mark.parametrize("mirror,name", [(_abi.ScanBwdArgs, "ssm_scan_bwd_args_t"),
                                         (_abi.CachedUpdateArgs, "ssm_cached_update_args_t")])
def test_struct_mirrors(tmp_path, mirror, name):
    fields = [f for f, _ in mirror._fields_]
    src = tmp_path / "o.c"
    src.write_text('#include <stdio.h>\n#include "ssm.h"\nint main(void) {\n' + "".join(
        f'printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) +
        f'printf("%zu\\n", sizeof({name}));\nreturn 0; }}\n')
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "o")])
    got = [int(v) for v in subprocess.check_output([str(tmp_path / "o")], text=True).split()]
    assert got == [getattr(mirror, f).offset for f in fields] + [ctypes.sizeof(mirror)]


def bwd(**kw):
    a = _abi.ScanBwdArgs()
    a.dtype, a.batch, a.dim, a.seqlen, a.dstate = 1, 2, 64, 128, 16
    for i, f in enumerate(["u", "delta", "A", "B", "C", "dout", "du", "ddelta", "dA", "dB", "dC", "workspace"]):
        setattr(a, f, FAKE + i * (1 << 28))
    a.workspace_bytes, a.delta_softplus = 1 << 27, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


P = FAKE + (40 << 28)
CASES = [
    (dict(dtype=3), "SSM_ERR_BAD_DTYPE"), (dict(batch=-1), "SSM_ERR_BAD_SHAPE"),
    (dict(dstate=0), "SSM_ERR_BAD_SHAPE"), (dict(dstate=129), "SSM_ERR_BAD_SHAPE"),
    (dict(a_heads=5), "SSM_ERR_BAD_SHAPE"), (dict(batch=70000), "SSM_ERR_UNSUPPORTED"),
    (dict(seqlen=1 << 30), "SSM_ERR_BAD_SHAPE"), (dict(dim=1 << 29, batch=60000), "SSM_ERR_BAD_SHAPE"),
    (dict(seqlen=1 << 29, dim=1 << 20), "SSM_ERR_BAD_SHAPE"), (dict(num_segments=-1), "SSM_ERR_BAD_SHAPE"),
    (dict(conv_weight=P, conv_width=5), "SSM_ERR_BAD_SHAPE"), (dict(conv_weight=P, conv_width=0), "SSM_ERR_BAD_SHAPE"),
    (dict(dconv_weight=P), "SSM_ERR_NULL_ARG"), (dict(conv_history=P), "SSM_ERR_NULL_ARG"),
    (dict(conv_weight=P, conv_width=4, dconv_history=P), "SSM_ERR_NULL_ARG"), (dict(dz=P), "SSM_ERR_NULL_ARG"),
    (dict(u_scale=P), "SSM_ERR_NULL_ARG"), (dict(u_scale=P, delta_scale=P, z=P), "SSM_ERR_NULL_ARG"),
    (dict(z=P, z_scale=P), "SSM_ERR_NULL_ARG"),
    (dict(reverse=1, initial_state=P), "SSM_ERR_UNSUPPORTED"), (dict(reverse=1, dinitial_state=P), "SSM_ERR_UNSUPPORTED"),
    (dict(seq_starts=P, num_seqs=1), "SSM_ERR_UNSUPPORTED"),
    (dict(seq_starts=P, num_seqs=0, batch=1), "SSM_ERR_BAD_SHAPE"),
    (dict(seq_starts=P, num_seqs=1, batch=1, dfinal_state=P), "SSM_ERR_UNSUPPORTED"),
    (dict(seq_starts=P, num_seqs=1, batch=1, reverse=1), "SSM_ERR_UNSUPPORTED"),
    (dict(seq_starts=P, num_seqs=1, batch=1, a_heads=2), "SSM_ERR_UNSUPPORTED"),
    (dict(channel_last=1, stride_u=63), "SSM_ERR_BAD_SHAPE"), (dict(channel_last=1, stride_dz=1 << 40), "SSM_ERR_BAD_SHAPE"),
    (dict(u=None), "SSM_ERR_NULL_ARG"), (dict(dA=None), "SSM_ERR_NULL_ARG"), (dict(dout=None), "SSM_ERR_NULL_ARG"),
    (dict(delta=FAKE + 1), "SSM_ERR_MISALIGNED"), (dict(dA=FAKE + 2), "SSM_ERR_MISALIGNED"),
    (dict(workspace=P + 8), "SSM_ERR_MISALIGNED"), (dict(workspace=None), "SSM_ERR_WORKSPACE"),
    (dict(workspace_bytes=100), "SSM_ERR_WORKSPACE"), (dict(du=FAKE), "SSM_ERR_ALIAS"),
    (dict(dB=FAKE + (3 << 28)), "SSM_ERR_ALIAS"), (dict(workspace=FAKE), "SSM_ERR_ALIAS"),
    (dict(dC=FAKE + (11 << 28)), "SSM_ERR_ALIAS"), (dict(ddelta=FAKE + (6 << 28)), "SSM_ERR_ALIAS"),
    # outputs that share some elements, dense or as columns of one tensor
    (dict(ddelta=FAKE + (6 << 28) + 64), "SSM_ERR_ALIAS"), (dict(dA=FAKE + (6 << 28) + 128), "SSM_ERR_ALIAS"),
    (dict(channel_last=1, stride_du=160, stride_ddelta=160, ddelta=FAKE + (6 << 28) + 126), "SSM_ERR_ALIAS"),
    (dict(channel_last=1, stride_du=160, stride_ddelta=160, ddelta=FAKE + (6 << 28) + 194), "SSM_ERR_ALIAS"),
    (dict(channel_last=1, stride_du=160, stride_ddelta=128, ddelta=FAKE + (6 << 28) + 128), "SSM_ERR_ALIAS"),
]


@pytest.mark.parametrize("kw,status", CASES)
def test_scan_bwd_refusals(lib, kw, status):
    assert _abi.STATUS[lib.ssm_selective_scan_bwd(ctypes.byref(bwd(**kw)), None)] == status
    assert lib.ssm_last_error_detail()


def test_null_args(lib):
    assert lib.ssm_selective_scan_bwd(None, None) == 1
    assert lib.ssm_selective_scan_bwd_workspace_size(ctypes.byref(bwd()), None) == 1
    assert lib.ssm_selective_state_update_cached(None, None) == 1


def test_workspace_sizes(lib):
    n = ctypes.c_size_t()

    def size(**kw):
        assert lib.ssm_selective_scan_bwd_workspace_size(ctypes.byref(bwd(workspace=None, **kw)), ctypes.byref(n)) == 0
        return n.value
    plain = size(num_segments=1)
    states = 2 * 64 * 128 // 8 * 16 * 4
    assert states <= plain <= 2 * states + (1 << 20)
    assert size(num_segments=1, conv_weight=P, conv_width=4) >= plain + 2 * 64 * 128 * 4
    assert size(num_segments=4) > plain
    assert size(seqlen=0) == 0 and size(batch=0) == 0
    # offsets and sizes past 32 bits
    assert size(batch=1, dim=5120, seqlen=1 << 20, num_segments=1) > 1 << 35
    assert lib.ssm_causal_conv1d_bwd_workspace_size(2, 3, 5000, ctypes.byref(n)) == 0
    rows, rest = divmod(n.value, 2 * 3 * 20)              # 5 fp32 sums per channel and piece of a row
    assert rest == 0 and 1 <= rows <= 5000
    assert _abi.STATUS[lib.ssm_causal_conv1d_bwd_workspace_size(-1, 3, 5, ctypes.byref(n))] == "SSM_ERR_BAD_SHAPE"


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), "SSM_ERR_BAD_DTYPE"), (dict(width=5), "SSM_ERR_BAD_SHAPE"), (dict(batch=-2), "SSM_ERR_BAD_SHAPE"),
    (dict(dout=None), "SSM_ERR_NULL_ARG"), (dict(dx=None), "SSM_ERR_NULL_ARG"), (dict(ws=None), "SSM_ERR_WORKSPACE"),
    (dict(ws_bytes=8), "SSM_ERR_WORKSPACE"), (dict(dx=FAKE), "SSM_ERR_ALIAS"), (dict(dx=FAKE + 1), "SSM_ERR_MISALIGNED"),
    (dict(dim=1 << 29, batch=1 << 20), "SSM_ERR_BAD_SHAPE"), (dict(dbias=FAKE + (4 << 28) + 64), "SSM_ERR_ALIAS"),
    (dict(dw=FAKE + (5 << 28)), "SSM_ERR_ALIAS"),
])
def test_conv_bwd_refusals(lib, kw, status):
    v = dict(dout=FAKE, x=FAKE + (1 << 28), w=FAKE + (2 << 28), bias=None, dx=FAKE + (3 << 28), dw=FAKE + (4 << 28),
             dbias=None, batch=2, dim=8, seqlen=100, width=4, silu=1, dtype=1, ws=FAKE + (5 << 28), ws_bytes=1 << 20)
    v.update(kw)
    assert _abi.STATUS[lib.ssm_causal_conv1d_bwd(*v.values(), None)] == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), "SSM_ERR_BAD_DTYPE"), (dict(seqlen=-1), "SSM_ERR_BAD_SHAPE"), (dict(batch=70000), "SSM_ERR_UNSUPPORTED"),
    (dict(x=None), "SSM_ERR_NULL_ARG"), (dict(codes=None), "SSM_ERR_NULL_ARG"), (dict(codes=FAKE), "SSM_ERR_ALIAS"),
    (dict(x=FAKE + 1), "SSM_ERR_MISALIGNED"), (dict(scales=FAKE + (2 << 28) + 2), "SSM_ERR_MISALIGNED"),
    (dict(cl=1, stride=7), "SSM_ERR_BAD_SHAPE"), (dict(seqlen=1 << 29, dim=1 << 29), "SSM_ERR_BAD_SHAPE"),
])
def test_pack_refusals(lib, kw, status):
    v = dict(x=FAKE, codes=FAKE + (1 << 28), scales=FAKE + (2 << 28), batch=2, dim=8, seqlen=100, cl=0, stride=0, dtype=1)
    v.update(kw)
    assert _abi.STATUS[lib.ssm_checkpoint_pack(*v.values(), None)] == status
    if "stride" not in kw:
        out = [v["codes"], v["scales"], v["x"], v["batch"], v["dim"], v["seqlen"], v["cl"], v["dtype"]]
        assert _abi.STATUS[lib.ssm_checkpoint_unpack(*out, None)] == status


def cached(**kw):
    a = _abi.CachedUpdateArgs()
    a.dtype, a.batch, a.dim, a.dstate, a.num_slots = 1, 2, 64, 16, 4
    for i, f in enumerate(["codes", "scales", "x", "dt", "A", "B_t", "C_t", "out"]):
        setattr(a, f, FAKE + i * (1 << 28))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), "SSM_ERR_BAD_DTYPE"), (dict(dstate=129), "SSM_ERR_BAD_SHAPE"), (dict(num_slots=1), "SSM_ERR_BAD_SHAPE"),
    (dict(num_slots=-1, slots=P), "SSM_ERR_BAD_SHAPE"), (dict(a_heads=3), "SSM_ERR_BAD_SHAPE"),
    (dict(conv_weight=P, conv_width=4), "SSM_ERR_NULL_ARG"), (dict(conv_weight=P, conv_width=6), "SSM_ERR_BAD_SHAPE"),
    (dict(codes=None), "SSM_ERR_NULL_ARG"), (dict(out=None), "SSM_ERR_NULL_ARG"), (dict(scales=FAKE + 2), "SSM_ERR_MISALIGNED"),
    (dict(out=FAKE + (2 << 28)), "SSM_ERR_ALIAS"), (dict(scales=FAKE), "SSM_ERR_ALIAS"),
    (dict(conv_weight=P, conv_width=4, conv_state=FAKE), "SSM_ERR_ALIAS"),
])
def test_cached_update_refusals(lib, kw, status):
    assert _abi.STATUS[lib.ssm_selective_state_update_cached(ctypes.byref(cached(**kw)), None)] == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), "SSM_ERR_BAD_SHAPE"), (dict(dstate=200), "SSM_ERR_BAD_SHAPE"), (dict(slots=None, num=1), "SSM_ERR_BAD_SHAPE"),
    (dict(state=None), "SSM_ERR_NULL_ARG"), (dict(codes=FAKE), "SSM_ERR_ALIAS"), (dict(scales=FAKE + (2 << 28) + 1), "SSM_ERR_MISALIGNED"),
])
def test_cache_refusals(lib, kw, status):
    v = dict(state=FAKE, codes=FAKE + (1 << 28), scales=FAKE + (2 << 28), slots=FAKE + (3 << 28), rand=None, batch=2, dim=8,
             dstate=16, num=4)
    v.update(kw)
    assert _abi.STATUS[lib.ssm_state_cache_write(*v.values(), None)] == status
    read = [v["codes"], v["scales"], v["slots"], v["state"], v["batch"], v["dim"], v["dstate"], v["num"], 0]
    assert _abi.STATUS[lib.ssm_state_cache_read(*read, None)] == status


def test_zero_sizes_launch_nothing(lib):
    """Nothing to do and nothing to point at: fine without a GPU."""
    assert lib.ssm_checkpoint_pack(None, None, None, 0, 8, 5, 0, 0, 1, None) == 0
    assert lib.ssm_state_cache_write(None, None, None, None, None, 0, 8, 16, 0, None) == 0
    assert lib.ssm_selective_state_update_cached(ctypes.byref(cached(batch=0)), None) == 0
