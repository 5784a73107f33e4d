"""What the bindings of the operators between the linears share: checks of
tensors, and the device and stream a call goes to."""
from __future__ import annotations

import ctypes

import torch

from . import _lib


def need(t, name: str, dtype, shape, device, contiguous: bool = True):
    """Raises ValueError unless t is a tensor of this type, shape and device
    (and contiguous)."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or (contiguous and not t.is_contiguous()):
        raise ValueError(f"{name} must be a {'contiguous ' if contiguous else ''}{dtype} {list(shape)} on {device}, "
                         f"not {t.dtype} {list(t.shape)} with strides {t.stride()} on {t.device}")


def rows(t, name: str, dtype, shape, device) -> int:
    """need() for a tensor whose dimensions after the first are contiguous;
    returns the first one's stride in elements."""
    need(t, name, dtype, shape, device, False)
    inner = 1
    for n, s in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and s != inner and t.numel() > 0:
            raise ValueError(f"every row of {name} must be contiguous (strides {t.stride()})")
        inner *= n
    return t.stride(0) if shape[0] > 1 else inner


def on_cuda(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def call(fn: str, device, stream, *args):
    """Calls the library's `fn` on `device` and its stream (the device's
    current stream when None), whatever the current device is."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"the tensors are on {device}, the stream on {stream.device}")
    f = getattr(_lib.load(), fn)
    if torch.cuda.current_device() == device.index:
        status = f(*args, ctypes.c_void_p(stream.cuda_stream))
    else:
        with torch.cuda.device(device):
            status = f(*args, ctypes.c_void_p(stream.cuda_stream))
    if status != _lib.OK:
        _lib._check(status, fn)


def ptr(t):
    return None if t is None else t.data_ptr()
