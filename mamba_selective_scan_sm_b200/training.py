"""Gradients of the selective scan and of the causal conv, and activations kept in 8 bits
between the forward and the backward pass (the training part of include/ssm.h)."""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import _abi
from ._marshal import DTYPES, Call, dtype_code, on_stream

__all__ = ["ScanGrads", "ConvGrads", "Packed8", "ssm_selective_scan_bwd",
           "ssm_selective_scan_bwd_workspace_size", "ssm_causal_conv1d_bwd",
           "ssm_checkpoint_pack", "ssm_checkpoint_unpack"]

BLOCK = 64                    # SSM_CHECKPOINT_BLOCK: positions of a channel per scale


class Packed8(NamedTuple):
    """An activation in 8 bits: int8 codes of its shape, and one fp32 scale per channel and
    64 positions, (batch, dim, nb) or channel-last (batch, nb, dim)."""
    codes: torch.Tensor
    scales: torch.Tensor


class ScanGrads(NamedTuple):
    """Gradients of ``ssm_selective_scan_fwd``'s inputs; None where the input was not given."""
    du: torch.Tensor
    ddelta: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddelta_bias: Optional[torch.Tensor]
    dconv_weight: Optional[torch.Tensor]
    dconv_bias: Optional[torch.Tensor]
    dinitial_state: Optional[torch.Tensor]
    dconv_history: Optional[torch.Tensor]


class ConvGrads(NamedTuple):
    """Gradients of ``ssm_causal_conv1d_fwd``'s inputs."""
    dx: torch.Tensor
    dw: torch.Tensor
    dbias: Optional[torch.Tensor]


def _blocks(seqlen):
    return -(-seqlen // BLOCK)


@functools.lru_cache(maxsize=256)
def _scan_workspace(dtype, batch, dim, seqlen, dstate, a_heads, conv_width, packed, channel_last,
                    num_segments):
    """The library's answer for these sizes (it depends on nothing else)."""
    lib = _abi.load()
    a = _abi.ScanBwdArgs()
    a.dtype, a.batch, a.dim, a.seqlen, a.dstate, a.a_heads = dtype, batch, dim, seqlen, dstate, a_heads
    a.conv_weight, a.conv_width = (1 if conv_width else None), conv_width
    a.seq_starts, a.num_seqs = (1, 1) if packed else (None, 0)
    a.channel_last, a.num_segments = channel_last, num_segments
    n = ctypes.c_size_t()
    _abi.check(lib, lib.ssm_selective_scan_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=256)
def _conv_workspace(batch, dim, seqlen):
    lib = _abi.load()
    n = ctypes.c_size_t()
    _abi.check(lib, lib.ssm_causal_conv1d_bwd_workspace_size(batch, dim, seqlen, ctypes.byref(n)))
    return n.value


def ssm_selective_scan_bwd_workspace_size(batch, dim, seqlen, dstate, dtype=torch.bfloat16, *,
                                          conv_width=0, a_heads=0, packed_sequences=False,
                                          channel_last=False, num_segments=0):
    """Workspace bytes ssm_selective_scan_bwd needs for these sizes (host-only query)."""
    if dtype not in DTYPES:
        raise TypeError(f"activations must be float32 or bfloat16, got {dtype}")
    return _scan_workspace(DTYPES[dtype], batch, dim, seqlen, dstate, a_heads, conv_width,
                           int(bool(packed_sequences)), int(bool(channel_last)), num_segments)


@on_stream
def ssm_selective_scan_bwd(dout, u, delta, A, B, C, D=None, z=None, delta_bias=None,
                           delta_softplus=True, reverse=False, conv_weight=None, conv_bias=None, *,
                           dfinal_state=None, initial_state=None, conv_history=None,
                           seq_starts=None, channel_last=False, du=None, ddelta=None, dz=None,
                           dB=None, dC=None, workspace=None, num_segments=0, stream=None):
    """Gradients of ``ssm_selective_scan_fwd(u, delta, A, B, C, ...)`` for the gradient
    ``dout`` of its output (and ``dfinal_state`` of its final state), from the forward call's
    inputs; arguments of the forward call's names are its arguments. B and C are
    input-dependent (3-D), the scan runs in one direction; the gradient of a bidirectional
    sum is the sum of two calls.

    ``u``, ``delta`` and ``z`` may be given as ``Packed8`` (all three): the gradients are
    then those of the values read back. ``du``, ``ddelta``, ``dz``, ``dB``, ``dC`` may be given
    as preallocated outputs (channel-last: views with a position stride, such as the halves
    of one in_proj gradient); ``workspace`` as uint8 scratch of at least
    ``ssm_selective_scan_bwd_workspace_size`` bytes. Returns ``ScanGrads``."""
    call = Call(dout)
    lib = _abi.load()
    a = _abi.ScanBwdArgs()
    a.dtype = dtype_code(dout, "dout")
    t, f32 = dout.dtype, torch.float32
    if dout.dim() != 3 or B.dim() != 3:
        raise ValueError("dout, B and C must have 3 axes")
    if channel_last:
        batch, seqlen, dim = dout.shape
        n = B.shape[2]
        shape, bc, sc = (batch, seqlen, dim), (batch, seqlen, n), (batch, _blocks(seqlen), dim)
    else:
        batch, dim, seqlen = dout.shape
        n = B.shape[1]
        shape, bc, sc = (batch, dim, seqlen), (batch, n, seqlen), (batch, dim, _blocks(seqlen))
    a.batch, a.dim, a.seqlen, a.dstate = batch, dim, seqlen, n
    a.channel_last = int(bool(channel_last))

    def act(x, name, shp, dt):
        """Pointer and stride of an activation-shaped tensor."""
        return call.strided(x, name, shp, dt) if channel_last else (call.ptr(x, name, shp, dt), 0)

    def kept(x, name):
        """(pointer, stride, scales) of an activation or of its 8-bit form."""
        if isinstance(x, Packed8):
            return (*act(x.codes, f"{name}.codes", shape, torch.int8),
                    call.ptr(x.scales, f"{name}.scales", sc, f32))
        return (*act(x, name, shape, t), None)

    given = [x for x in (u, delta, z) if x is not None]
    if any(isinstance(x, Packed8) for x in given) and not all(isinstance(x, Packed8) for x in given):
        raise TypeError("u, delta and z are all Packed8 or none")
    a.u, a.stride_u, a.u_scale = kept(u, "u")
    a.delta, a.stride_delta, a.delta_scale = kept(delta, "delta")
    a.z, a.stride_z, a.z_scale = kept(z, "z")
    a.B, a.stride_B = act(B, "B", bc, t)
    a.C, a.stride_C = act(C, "C", bc, t)
    a.dout, a.stride_dout = act(dout, "dout", shape, t)
    a.a_heads = A.shape[0] if A.dim() == 1 else 0
    a.A = call.ptr(A, "A", (A.shape[0],) if A.dim() == 1 else (dim, n), f32)
    a.D = call.ptr(D, "D", (dim,), f32)
    a.delta_bias = call.ptr(delta_bias, "delta_bias", (dim,), f32)
    a.delta_softplus, a.reverse = int(bool(delta_softplus)), int(bool(reverse))
    width = 0
    if conv_weight is not None:
        width = conv_weight.shape[-1]
        if width < 1:
            raise ValueError("conv_weight has no taps")
        a.conv_weight, a.conv_width = call.ptr(conv_weight, "conv_weight", (dim, width), f32), width
        a.conv_bias = call.ptr(conv_bias, "conv_bias", (dim,), f32)
    elif conv_bias is not None or conv_history is not None:
        raise ValueError("conv_bias and conv_history need conv_weight")
    state, hist = (batch, dim, n), (batch, dim, max(width - 1, 0))
    a.initial_state = call.ptr(initial_state, "initial_state", state, f32)
    a.dfinal_state = call.ptr(dfinal_state, "dfinal_state", state, f32)
    a.conv_history = call.ptr(conv_history, "conv_history", hist, t)
    if seq_starts is not None:
        if seq_starts.dim() != 1 or seq_starts.numel() < 2:
            raise ValueError("seq_starts must hold num_seqs + 1 offsets")
        a.num_seqs = seq_starts.numel() - 1
        a.seq_starts = call.ptr(seq_starts, "seq_starts", (a.num_seqs + 1,), torch.int32)
    a.num_segments = int(num_segments)

    def new(shp, dt=f32):
        return torch.empty(shp, dtype=dt, device=call.device)

    du = new(shape, t) if du is None else du
    ddelta = new(shape, t) if ddelta is None else ddelta
    dB = new(bc, t) if dB is None else dB
    dC = new(bc, t) if dC is None else dC
    if z is None and dz is not None:
        raise ValueError("dz needs z")
    dz = new(shape, t) if dz is None and z is not None else dz
    g = ScanGrads(
        du, ddelta, torch.empty_like(A), dB, dC, None if D is None else torch.empty_like(D), dz,
        None if delta_bias is None else torch.empty_like(delta_bias),
        None if conv_weight is None else torch.empty_like(conv_weight),
        None if conv_bias is None else torch.empty_like(conv_bias),
        None if initial_state is None else torch.empty_like(initial_state),
        None if conv_history is None else torch.empty_like(conv_history))
    a.du, a.stride_du = act(du, "du", shape, t)
    a.ddelta, a.stride_ddelta = act(ddelta, "ddelta", shape, t)
    a.dz, a.stride_dz = act(dz, "dz", shape, t)
    a.dB, a.stride_dB = act(dB, "dB", bc, t)
    a.dC, a.stride_dC = act(dC, "dC", bc, t)
    for name in ("dA", "dD", "ddelta_bias", "dconv_weight", "dconv_bias", "dinitial_state",
                 "dconv_history"):
        v = getattr(g, name)
        setattr(a, name, None if v is None else v.data_ptr() or None)
    need = _scan_workspace(a.dtype, batch, dim, seqlen, n, a.a_heads, width, int(seq_starts is not None),
                           a.channel_last, a.num_segments)
    if need:
        if workspace is None:
            workspace = new(need, torch.uint8)
        else:
            call.ptr(workspace, "workspace", workspace.shape, torch.uint8)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    call.run(lib.ssm_selective_scan_bwd, (ctypes.byref(a),), stream)
    return g


@on_stream
def ssm_causal_conv1d_bwd(dout, x, w, bias=None, apply_silu=True, *, workspace=None, stream=None):
    """Gradients of ``ssm_causal_conv1d_fwd(x, w, bias, apply_silu)`` for the gradient
    ``dout`` of its output. Returns ``ConvGrads(dx, dw, dbias)``."""
    call = Call(dout)
    lib = _abi.load()
    code = dtype_code(dout, "dout")
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be (batch, dim, seqlen) and w (dim, width)")
    batch, dim, seqlen = x.shape
    width = w.shape[1]
    px = call.ptr(x, "x", x.shape, dout.dtype)
    pd = call.ptr(dout, "dout", x.shape, dout.dtype)
    pw = call.ptr(w, "w", (dim, width), torch.float32)
    pb = call.ptr(bias, "bias", (dim,), torch.float32)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db = None if bias is None else torch.empty_like(bias)
    if workspace is None:
        workspace = torch.empty(_conv_workspace(batch, dim, seqlen), dtype=torch.uint8, device=call.device)
    else:
        call.ptr(workspace, "workspace", workspace.shape, torch.uint8)
    call.run(lib.ssm_causal_conv1d_bwd,
             (pd, px, pw, pb, dx.data_ptr() or None, dw.data_ptr() or None,
              None if db is None else db.data_ptr() or None, batch, dim, seqlen, width,
              int(bool(apply_silu)), code, workspace.data_ptr() or None, workspace.numel()), stream)
    return ConvGrads(dx, dw, db)


@on_stream
def ssm_checkpoint_pack(x, *, channel_last=False, codes=None, scales=None, stream=None):
    """Pack an activation into 8 bits: x (batch, dim, seqlen), or channel-last (batch,
    seqlen, dim), possibly a view with a position stride. Per channel and 64 positions,
    code = round(127 x / max|x|) and scale = max|x| / 127. Returns ``Packed8``."""
    call = Call(x)
    lib = _abi.load()
    code = dtype_code(x, "x")
    if x.dim() != 3:
        raise ValueError("x must have 3 axes")
    if channel_last:
        batch, seqlen, dim = x.shape
        ptr, step = call.strided(x, "x", x.shape, x.dtype)
        sc = (batch, _blocks(seqlen), dim)
    else:
        batch, dim, seqlen = x.shape
        ptr, step = call.ptr(x, "x", x.shape, x.dtype), 0
        sc = (batch, dim, _blocks(seqlen))
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.int8, device=call.device)
    if scales is None:
        scales = torch.empty(sc, dtype=torch.float32, device=call.device)
    call.run(lib.ssm_checkpoint_pack,
             (ptr, call.ptr(codes, "codes", x.shape, torch.int8),
              call.ptr(scales, "scales", sc, torch.float32), batch, dim, seqlen,
              int(bool(channel_last)), step, code), stream)
    return Packed8(codes, scales)


@on_stream
def ssm_checkpoint_unpack(packed, dtype=torch.bfloat16, *, channel_last=False, out=None, stream=None):
    """Read a ``Packed8`` back as a dense tensor of ``dtype`` (or into ``out``)."""
    codes, scales = packed
    call = Call(codes)
    lib = _abi.load()
    if codes.dim() != 3:
        raise ValueError("codes must have 3 axes")
    if channel_last:
        batch, seqlen, dim = codes.shape
        sc = (batch, _blocks(seqlen), dim)
    else:
        batch, dim, seqlen = codes.shape
        sc = (batch, dim, _blocks(seqlen))
    if out is None:
        out = torch.empty(codes.shape, dtype=dtype, device=call.device)
    call.run(lib.ssm_checkpoint_unpack,
             (call.ptr(codes, "codes", codes.shape, torch.int8),
              call.ptr(scales, "scales", sc, torch.float32),
              call.ptr(out, "out", codes.shape, out.dtype), batch, dim, seqlen,
              int(bool(channel_last)), dtype_code(out, "out")), stream)
    return out
