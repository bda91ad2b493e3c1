"""Decode states in 8 bits (the cache part of include/ssm.h): a cache is a pair of tensors,
``codes`` int8 (num_slots, dim, dstate) and ``scales`` fp32 (num_slots, dim), that the caller
allocates and keeps. ``slots`` (int32, one per batch row) says which slot a row uses; a row
whose slot is negative or past the end is padding, and its outputs are left as they were.
``rand`` (int32 or uint32 bits, (batch, dim)) rounds at random instead of to the nearest."""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._marshal import Call, dtype_code, on_stream

__all__ = ["ssm_state_cache_write", "ssm_state_cache_read", "ssm_selective_state_update_cached"]


def _cache(call, codes, scales, slots, rand, batch):
    """Checked pointers of the cache and of what selects and rounds its rows."""
    if codes.dim() != 3:
        raise ValueError("codes must be (num_slots, dim, dstate)")
    num_slots, dim, _ = codes.shape
    if rand is not None and rand.dtype not in (torch.int32, torch.uint32):
        raise TypeError("rand must be int32 or uint32")
    return (call.ptr(codes, "codes", codes.shape, torch.int8),
            call.ptr(scales, "scales", (num_slots, dim), torch.float32),
            call.ptr(slots, "slots", (batch,), torch.int32),
            call.ptr(rand, "rand", (batch, dim), rand.dtype if rand is not None else None))


@on_stream
def ssm_state_cache_write(state, codes, scales, *, slots=None, rand=None, stream=None):
    """Write fp32 states (batch, dim, dstate) into their slots of the cache."""
    call = Call(codes)
    lib = _abi.load()
    batch = state.shape[0]
    pc, ps, psl, pr = _cache(call, codes, scales, slots, rand, batch)
    num_slots, dim, n = codes.shape
    call.run(lib.ssm_state_cache_write,
             (call.ptr(state, "state", (batch, dim, n), torch.float32), pc, ps, psl, pr, batch, dim,
              n, num_slots), stream)


@on_stream
def ssm_state_cache_read(codes, scales, *, slots=None, dtype=torch.float32, out=None, stream=None):
    """The states of the slots, (batch, dim, dstate) in ``dtype`` (or into ``out``, whose rows
    without a slot keep what they hold; a new tensor has zeros there)."""
    call = Call(codes)
    lib = _abi.load()
    batch = slots.shape[0] if slots is not None else codes.shape[0]
    pc, ps, psl, _ = _cache(call, codes, scales, slots, None, batch)
    num_slots, dim, n = codes.shape
    if out is None:
        make = torch.empty if slots is None else torch.zeros
        out = make(batch, dim, n, dtype=dtype, device=call.device)
    call.run(lib.ssm_state_cache_read,
             (pc, ps, psl, call.ptr(out, "out", (batch, dim, n), out.dtype), batch, dim, n,
              num_slots, dtype_code(out, "out")), stream)
    return out


@on_stream
def ssm_selective_state_update_cached(codes, scales, conv_state, x, dt, A, B, C, D=None, z=None,
                                      dt_bias=None, dt_softplus=True, conv_weight=None,
                                      conv_bias=None, *, slots=None, rand=None, out=None,
                                      stream=None):
    """One decode step (``ssm_selective_state_update``) on a cache of states in 8 bits, in
    place on ``codes``, ``scales`` and ``conv_state`` (num_slots, dim, width). x, dt, z
    (batch, dim); B, C (batch, dstate); A (dim, dstate), or (nheads,) for one scalar per
    head. The output comes from the new state before it is rounded. Returns y (batch, dim);
    a new tensor has zeros in the rows without a slot."""
    call = Call(codes)
    lib = _abi.load()
    a = _abi.CachedUpdateArgs()
    a.dtype = dtype_code(x, "x")
    batch, t, f32 = x.shape[0], x.dtype, torch.float32
    a.codes, a.scales, a.slots, a.rand = _cache(call, codes, scales, slots, rand, batch)
    num_slots, dim, n = codes.shape
    a.batch, a.dim, a.dstate, a.num_slots = batch, dim, n, num_slots
    row, bc = (batch, dim), (batch, n)
    a.x, a.dt, a.z = call.ptr(x, "x", row, t), call.ptr(dt, "dt", row, t), call.ptr(z, "z", row, t)
    a.B_t, a.C_t = call.ptr(B, "B", bc, t), call.ptr(C, "C", bc, t)
    a.a_heads = A.shape[0] if A.dim() == 1 else 0
    a.A = call.ptr(A, "A", (A.shape[0],) if A.dim() == 1 else (dim, n), f32)
    a.D = call.ptr(D, "D", (dim,), f32)
    a.dt_bias, a.dt_softplus = call.ptr(dt_bias, "dt_bias", (dim,), f32), int(bool(dt_softplus))
    if conv_weight is not None:
        width = conv_weight.shape[-1]
        if width < 1:
            raise ValueError("conv_weight has no taps")
        a.conv_weight, a.conv_width = call.ptr(conv_weight, "conv_weight", (dim, width), f32), width
        a.conv_bias = call.ptr(conv_bias, "conv_bias", (dim,), f32)
        if conv_state is None:
            raise ValueError("conv_weight needs conv_state")
        a.conv_state = call.ptr(conv_state, "conv_state", (num_slots, dim, width), t)
    elif conv_bias is not None:
        raise ValueError("conv_bias needs conv_weight")
    if out is None:
        out = (torch.empty if slots is None else torch.zeros)(batch, dim, dtype=t, device=call.device)
    a.out = call.ptr(out, "out", row, t)
    call.run(lib.ssm_selective_state_update_cached, (ctypes.byref(a),), stream)
    return out
