"""Tensor arguments of the C ABI's calls: their checks, pointers and streams."""
from __future__ import annotations

import contextlib

import torch


def _ptr(t: torch.Tensor | None) -> int:
    # a plain int: the entry points' argtypes make it a void*
    return 0 if t is None else t.data_ptr()


def _stream(stream: torch.cuda.Stream | None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the current stream's handle, without building a Stream object per call
    # where torch offers that
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


_current = contextlib.nullcontext()


def _on(stream: torch.cuda.Stream | None):
    """A context in which `stream` is the current stream; None changes nothing."""
    return _current if stream is None else torch.cuda.stream(stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _need(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str, cuda: bool = True) -> None:
    # one cheap test on the common path; the detailed ones only on failure
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_cuda is cuda and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} must be a host tensor")
