"""What the bindings of the operators between the linears share: checks of
tensors, and the device and stream a call goes to.  A decode step makes a few
such calls per layer, so they are kept short."""
from __future__ import annotations

from contextlib import nullcontext

import torch

from . import _lib

_functions = {}


def need(t, name: str, dtype, shape, device: int):
    """Raises ValueError unless t is a contiguous tensor of this type and shape
    on this CUDA device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} on cuda:{device}, "
                         f"not {t.dtype} {list(t.shape)} with strides {t.stride()} on {t.device}")


def rows(t, name: str, dtype, shape, device: int) -> int:
    """need() for a tensor whose first dimension may have any stride; returns
    that stride in elements."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name} must be a {dtype} {list(shape)} on cuda:{device}, "
                         f"not {t.dtype} {list(t.shape)} on {t.device}")
    strides = t.stride()
    n = len(strides)
    if n == 3 and strides[2] == 1 and strides[1] == shape[2] and shape[0] > 1 or n == 2 and strides[1] == 1 and shape[0] > 1:
        return strides[0]
    inner = 1
    for i in range(len(shape) - 1, 0, -1):
        if strides[i] != inner and shape[i] != 1 and t.numel() > 0:
            raise ValueError(f"every row of {name} must be contiguous (strides {strides})")
        inner *= shape[i]
    return strides[0] if shape[0] > 1 else inner


def on_cuda(t, name: str) -> int:
    """The index of the CUDA device that t is on."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def call(fn: str, device: int, stream, *args):
    """Calls the library's `fn` on the CUDA device and its stream (the device's
    current one when None), whatever the current device is."""
    f = _functions.get(fn)
    if f is None:
        f = _functions[fn] = getattr(_lib.load(), fn)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device)
    elif stream.device.index != device:
        raise ValueError(f"the tensors are on cuda:{device}, the stream on {stream.device}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == device:
        status = f(*args, handle)
    else:
        with torch.cuda.device(device):
            status = f(*args, handle)
    if status != _lib.OK:
        _lib._check(status, fn)


def allocating(stream):
    """A context in which new tensors belong to `stream` (the current one when
    None): what fills them comes before the call's kernels there, and their
    memory goes to others only behind them."""
    return nullcontext() if stream is None else torch.cuda.stream(stream)


def ptr(t):
    return None if t is None else t.data_ptr()
