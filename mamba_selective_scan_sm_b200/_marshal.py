"""Argument checks shared by the training and cache bindings: shapes, types and devices are
checked here (ValueError / TypeError), sizes and pointers in the library (SSMError)."""
from __future__ import annotations

import ctypes

import torch

from . import _abi

DTYPES = {torch.float32: _abi.SSM_F32, torch.bfloat16: _abi.SSM_BF16}


def dtype_code(t, name="activations"):
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return DTYPES[t.dtype]


class Call:
    """The tensors of one call: all on one device, each of its shape and type."""

    def __init__(self, first):
        if not first.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        self.device = first.device

    def ptr(self, t, name, shape, dtype):
        """A contiguous tensor's pointer (None for None or an empty one)."""
        self.check(t, name, shape, dtype)
        if t is None:
            return None
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr() or None

    def check(self, t, name, shape, dtype):
        if t is None:
            return
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, not on {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")

    def strided(self, t, name, shape, dtype):
        """(pointer, position stride) of a channel-last (batch, seqlen, width) view: its last
        axis dense, its batch rows seqlen positions apart."""
        self.check(t, name, shape, dtype)
        if t is None or not t.numel():
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
        if stream is not None and stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {self.device}")
        with torch.cuda.device(self.device):
            s = torch.cuda.current_stream() if stream is None else stream
            _abi.check(_abi.load(), fn(*args, ctypes.c_void_p(s.cuda_stream)))
