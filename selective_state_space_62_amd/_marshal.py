"""What the tensor-level calls of the recurrence and of the rotation share: cheap checks, addresses,
workspaces and the launch on torch's current stream.  A call's host time is most of a small call."""
from __future__ import annotations

import torch

from .binding import _check
from .torch_ops import _IO, _need

current_device = torch._C._cuda_getDevice
current_stream = torch._C._cuda_getCurrentRawStream   # the stream's address, without a Stream object


def io_code(t, name):
    """The library's code of a tensor's I/O type, that type, and the tensor's device, a GPU."""
    dtype = t.dtype
    io = _IO.get(dtype)
    if io is None:
        raise TypeError("%s must be float32 or bfloat16" % name)
    if not t.is_cuda:
        raise ValueError("inputs must be on a GPU")
    return io, dtype, t.device


def need(named, dtype, shape, device):
    """Every tensor of the (name, tensor or None) pairs has this type, shape and device and is contiguous."""
    for name, t in named:
        if t is not None and (t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous()):
            _need(t, name, dtype, shape, device)   # says which


def ptr(t):
    return None if t is None else t.data_ptr()


def workspace(given, nbytes, device):
    """(tensor to keep, address, bytes) of the caller's workspace, or of a new one; nothing where none is needed."""
    if given is None:
        if not nbytes:
            return None, None, 0
        given = torch.empty(nbytes, dtype=torch.uint8, device=device)
        return given, given.data_ptr(), nbytes
    have = given.numel() * given.element_size()
    if have < nbytes:
        raise ValueError("workspace has %d bytes, %d needed" % (have, nbytes))
    if given.device != device or not given.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % (device,))
    return given, given.data_ptr(), have


def launch(device, fn, *args):
    """fn(*args, stream), of the library, on torch's current stream of `device`, which is made the current device for it."""
    index = device.index
    if index == current_device():
        status = fn(*args, current_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, current_stream(index))
    if status:
        _check(status)
