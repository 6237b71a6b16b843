"""Argument checks and launch context of the entry points that also serve single tokens, where the
call itself counts: the common case costs one comparison of each property."""
from __future__ import annotations

import contextlib

import torch

from .wkv7 import _check

_here = contextlib.nullcontext()


def expect(t, name, dtype, shape, like):
    """t is a dense CUDA tensor of that type and shape on the device of `like`."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.device == like.device
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    _check(t, name, dtype, shape)
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, the call on {like.device}: one device only")


def address(t):
    return None if t is None else t.data_ptr()


def on_device(t):
    """A context with t's device current (nothing to do where it is)."""
    return _here if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)


def stream(t) -> int:
    """The current stream of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)
