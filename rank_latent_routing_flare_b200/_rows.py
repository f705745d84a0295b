"""Helpers of the operators of include/flare_ops.h: checks of [B, H, N, D]
tensors of rows and the packing of argument structs (every member 8 bytes)."""
from __future__ import annotations

import torch

from . import _binding as b

ROW_WIDTHS = (16, 32, 64, 128)


def check_rows(name, t, shape, output=False):
    """bf16 CUDA tensor of that shape, dense along D, rows on 16-byte boundaries."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    sb, sh, sn, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must be dense along its last dimension")
    if t.data_ptr() & 15 or any(s & 7 for s, n in zip((sb, sh, sn), shape) if n > 1):
        raise ValueError(f"{name}: every row must start on a 16-byte boundary (strides {t.stride()})")
    if output and any(s == 0 for s, n in zip((sb, sh, sn), shape) if n > 1):
        raise ValueError(f"{name} is written and must not be an expanded view")


def check_small(name, t, dtype, shape, device):
    """Optional contiguous tensor on the operator's device."""
    if t is None:
        return
    b._check_dev(name, t, dtype, shape)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def rows(t):
    """Pointer and the three strides of a tensor of rows, as the argument structs hold them."""
    if t is None:
        return 0, 0, 0, 0
    s = t.stride()
    return t.data_ptr(), s[0], s[1], s[2]


def call(fn, where, device, stream, *args):
    """fn(*args, stream) with `device` current; raises FlareError on a status other than OK."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"{where}: the stream is on {stream.device}, the tensors on {device}")
    if torch.cuda.current_device() == device.index:
        st = fn(*args, stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream.cuda_stream)
    if st != 0:
        raise b.FlareError(st, where)


def workspace(ws, nbytes, device):
    if ws is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    check_small("workspace", ws, torch.uint8, None, device)
    if ws.numel() < nbytes:
        raise ValueError(f"workspace has {ws.numel()} bytes, needs {nbytes}")
    return ws
