"""What the bindings of the small operators share: tensor checks, device and stream of a
call, workspaces.  A call of a few microseconds on the GPU is bound by the host, so a
tensor that is as it should be costs one expression here; only a wrong one goes through
``api._need``, which words the error."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from .api import _need

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def need(t: torch.Tensor, name: str, dtype, dev: torch.device, shape) -> int:
    """The address of t, which has to be a contiguous tensor of that type, device and shape."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.device == dev
            and t.shape == shape and t.is_contiguous()):
        _need(t, name, dtype, dev, shape)
    return t.data_ptr()


def maybe(t: Optional[torch.Tensor], name: str, dtype, dev: torch.device, shape) -> Optional[int]:
    return None if t is None else need(t, name, dtype, dev, shape)


def size(func: str, *args) -> int:
    """What a workspace query answers."""
    n = ctypes.c_size_t(0)
    _lib.check(getattr(_lib.load(), func)(*args, ctypes.byref(n)), func)
    return n.value


def scratch(workspace: Optional[torch.Tensor], bytes_needed: int, dev: torch.device
            ) -> Optional[torch.Tensor]:
    """The caller's workspace, or one from torch's allocator."""
    if workspace is None:
        return torch.empty(bytes_needed, device=dev, dtype=torch.uint8) if bytes_needed else None
    _need(workspace, "workspace", torch.uint8, dev)
    if workspace.numel() < bytes_needed:
        raise ValueError(f"workspace has {workspace.numel()} bytes, {bytes_needed} needed")
    return workspace


def call(func: str, dev: torch.device, *args) -> None:
    """func(*args, stream) on dev's current stream, with dev current."""
    index = dev.index
    if index == torch.cuda.current_device():
        stream = (_raw_stream(index) if _raw_stream is not None
                  else torch.cuda.current_stream(dev).cuda_stream)
        status = getattr(_lib.load(), func)(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = getattr(_lib.load(), func)(*args,
                                                torch.cuda.current_stream(dev).cuda_stream)
    if status:
        _lib.check(status, func)
