"""Argument checks shared by the training and cache bindings: shapes, types and devices are
checked here (ValueError / TypeError), sizes and pointers in the library (SSMError)."""
from __future__ import annotations

import functools

import torch

from . import _abi

DTYPES = {torch.float32: _abi.SSM_F32, torch.bfloat16: _abi.SSM_BF16}


def dtype_code(t, name="activations"):
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return DTYPES[t.dtype]


def on_stream(fn):
    """Run a call that is given a stream with that stream current, so that what it allocates
    (outputs, workspace) belongs to the stream that uses it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, stream=stream, **kw)
    return call


class Call:
    """The tensors of one call: all on one device, each of its shape and type."""

    def __init__(self, first):
        if not first.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        self.device = first.device

    def ptr(self, t, name, shape, dtype):
        """A contiguous tensor's pointer (None for None or an empty one)."""
        if t is None:
            return None
        self.check(t, name, shape, dtype)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr() or None

    def check(self, t, name, shape, dtype):
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, not on {self.device}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")

    def strided(self, t, name, shape, dtype):
        """(pointer, position stride) of a channel-last (batch, seqlen, width) view: its last
        axis dense, its batch rows seqlen positions apart."""
        if t is None:
            return None, 0
        self.check(t, name, shape, dtype)
        if not t.numel():
            return None, 0
        b, length, w = shape
        if w > 1 and t.stride(2) != 1:
            raise ValueError(f"{name}: channel-last views need a dense last axis")
        if length > 1:
            step = t.stride(1)
        else:
            step = t.stride(0) if b > 1 else w
        if (b > 1 and t.stride(0) != length * step) or (b * length > 1 and step < w):
            raise ValueError(f"{name}: channel-last views need stride (seqlen*s, s, 1), s >= width")
        return t.data_ptr(), step

    def run(self, fn, args, stream):
        """Call the library with the tensors' device current, on `stream` or that device's
        current stream."""
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {self.device}")
        if torch.cuda.current_device() == self.device.index:
            status = fn(*args, stream.cuda_stream)
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, stream.cuda_stream)
        if status:
            _abi.check(_abi.load(), status)
