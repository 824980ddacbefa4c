"""Checks and guards of the wrappers that take torch tensors."""
from __future__ import annotations

import contextlib

import torch

from . import capi

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # 2 us less than a Stream
current_device = torch.cuda.current_device


def check_tensor(t, name: str, dtype, shape=None, device=None) -> None:
    """`t` is a contiguous CUDA tensor of this type, shape and device."""
    if t.dtype != dtype or (shape is not None and t.shape != shape) or not t.is_contiguous() \
            or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be contiguous {dtype}"
                         + (f" of shape {tuple(shape)}" if shape is not None else "")
                         + f" on {device or 'a CUDA device'}, got {t.dtype} {tuple(t.shape)} with "
                         f"strides {t.stride()} on {t.device}")


def check_heads(t: torch.Tensor, name: str, device):
    """The shape of a tensor [tokens, heads, head_dim] with contiguous heads."""
    if t.dim() != 3 or t.device != device:
        raise ValueError(f"{name} must be [tokens, heads, head_dim] on {device}")
    shape, stride = t.shape, t.stride()
    if stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{name} must have contiguous heads, got strides {stride}")
    return shape


def same_device(device, **tensors) -> None:
    if device.type != "cuda":
        raise ValueError(f"a CUDA device is needed, got {device}")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def dtype_code(t, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return capi.DEC_BF16
    if t.dtype == torch.float32:
        return capi.DEC_F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")


class guard:
    """Makes `device`, and `stream` if it is not None, current: kernels run
    there and scratch allocated within belongs to that stream."""

    def __init__(self, device, stream):
        on = getattr(stream, "device", None)   # (a raw or foreign handle is taken to be of `device`)
        if isinstance(on, torch.device) and on != device:
            raise ValueError(f"the stream must be one of {device}, got one of {on}")
        self.device, self.stream = device, stream

    def __enter__(self):
        self.stack = contextlib.ExitStack()
        self.stack.enter_context(torch.cuda.device(self.device))
        if self.stream is not None:
            s = self.stream
            if not isinstance(s, torch.cuda.Stream):
                s = torch.cuda.ExternalStream(int(getattr(s, "cuda_stream", s)), device=self.device)
            self.stack.enter_context(torch.cuda.stream(s))

    def __exit__(self, *exc):
        return self.stack.__exit__(*exc)


def elsewhere(device, stream) -> bool:
    """Whether a call on `device` and `stream` (None: the current one) needs a
    guard before it can use current_stream_of()."""
    return stream is not None or current_device() != device.index


def current_stream_of(device) -> int:
    """The raw current stream of `device`."""
    return _raw_stream(device.index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
