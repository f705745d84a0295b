"""Helpers of the operators of include/flare_ops.h: checks of [B, H, N, D]
tensors of rows and the packing of argument structs (every member 8 bytes).

A call on a few rows takes a few microseconds on the GPU, so the checks read
each tensor's properties once and hand back what the struct needs.
"""
from __future__ import annotations

import functools

import torch

from . import _binding as b

ROW_WIDTHS = (16, 32, 64, 128)
NO_ROWS = (0, 0, 0, 0)
_bf16, _dense, empty_like = torch.bfloat16, torch.contiguous_format, torch.empty_like


def rows(t):
    """Pointer and the three strides of a tensor of rows, as the argument structs hold them."""
    return (t.data_ptr(), *t.stride()[:3])


def check_rows(name, t, shape, dev, output=False):
    """Checks a bf16 tensor of that shape on GPU `dev`, dense along D, its rows
    on 16-byte boundaries; returns its pointer and strides."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not _bf16 or t.shape != shape:
        _refuse(name, t, _bf16, shape, dev)
    p, (sb, sh, sn, sd) = t.data_ptr(), t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError(f"{name} must be dense along its last dimension")
    if p & 15 or (sb | sh | sn) & 7:
        if p & 15 or any(s & 7 for s, n in zip((sb, sh, sn), shape) if n > 1):
            raise ValueError(f"{name}: every row must start on a 16-byte boundary (strides {t.stride()})")
    if output and not (sb and sh and sn) and any(s == 0 for s, n in zip((sb, sh, sn), shape) if n > 1):
        raise ValueError(f"{name} is written and must not be an expanded view")
    return p, sb, sh, sn


def check_small(name, t, dtype, shape, dev) -> int:
    """Checks a contiguous tensor on GPU `dev` (shape None: any); returns its pointer."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype or (
            shape is not None and t.shape != shape):
        _refuse(name, t, dtype, shape, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _refuse(name, t, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def no_gradient(what, **tensors):
    """Refuses tensors that ask for a gradient which is not computed, where gradients are recorded."""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if t is not None and t.requires_grad:
                raise ValueError(f"{name}: gradients with respect to the {what} are not computed")


def dense(t):
    """A gradient as rows that the kernels can read: autograd may hand over fp32
    tensors, expanded ones, and dense views at any offset of a larger one."""
    t = t.to(_bf16).contiguous()
    return t.clone() if t.data_ptr() & 15 else t


def ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


@functools.lru_cache(maxsize=None)
def entry(name):
    """Entry point of the library."""
    return getattr(b.load_library(), name)


def call(name, where, dev, stream, *args):
    """The entry point called with GPU `dev` current, on `stream` (None: the
    current one); raises FlareError on a status other than OK."""
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"{where}: the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        s = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = entry(name)(*args, s)
    else:
        with torch.cuda.device(dev):
            st = entry(name)(*args, s)
    if st != 0:
        raise b.FlareError(st, where)


# What a call allocates for work on another stream than the current one comes
# from that stream's memory: a block that was freed on the current one may still
# be read by work queued there.  Outputs are recorded on the current stream,
# where the caller goes on with them.

def new(make, stream):
    """make(), a new output of a call on `stream` (None: the current one)."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def new_like(like, stream):
    return new(lambda: empty_like(like, memory_format=_dense), stream)


def output(name, t, like, dev, stream, check):
    """An output of `like`'s shape, new unless given, and its pointer and strides."""
    if t is None:
        t = empty_like(like, memory_format=_dense) if stream is None else new_like(like, stream)
    elif check:
        return t, check_rows(name, t, like.shape, dev, output=True)
    return (t, (t.data_ptr(), *t.stride()[:3]))


def workspace(ws, nbytes, like, stream):
    """The caller's workspace, checked, or a new one."""
    if ws is None:
        if stream is not None:
            with torch.cuda.stream(stream):
                return workspace(None, nbytes, like, None)
        return torch.empty(nbytes if nbytes > 256 else 256, dtype=torch.uint8, device=like.device)
    check_small("workspace", ws, torch.uint8, None, like.get_device())
    if ws.numel() < nbytes:
        raise ValueError(f"workspace has {ws.numel()} bytes, needs {nbytes}")
    return ws
