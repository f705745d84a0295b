"""Exact softmax attention: capped scores, a distance bias, and causal, prefix,
packed-document and padding masks; forward, backward, and single new tokens
over a cache.

The N x N attention that the mixer approximates through its latents, on the
same [B, H, N, D] tensors (any strides with dense rows).  Argument checks and
marshalling only: the kernels are behind include/flare_ops.h.
"""
from __future__ import annotations

import functools
import struct

import torch
from torch.autograd.function import once_differentiable

from . import _binding as b
from ._rows import (NO_ROWS, ROW_WIDTHS, call, check_rows, check_small, dense, entry, new, no_gradient,
                    output as _output, ptr, rows, workspace as _ws)

# flare_attention_args
_ARGS = struct.Struct("=7q2d12q6q4qq4q12q")
_f32, _i32 = torch.float32, torch.int32
_NO_BACKWARD = NO_ROWS * 4


@functools.lru_cache(maxsize=4096)
def flare_attention_workspace_bytes(B: int, Hq: int, Hk: int, Nq: int, Nk: int, D: int, backward: bool = False) -> int:
    return int(entry("flare_attention_workspace_bytes")(B, Hq, Hk, Nq, Nk, D, int(backward)))


def _head(Q, K, V, lengths, q_lengths, q_offsets, documents, prefix, slopes, causal, scale, cap, check):
    """The inputs' part of the argument struct, in its order, and the sizes with the device index."""
    if Q.dim() != 4 or K.dim() != 4 or V.dim() != 4:
        raise ValueError("Q, K and V are [B, H, N, D]")
    B, Hq, Nq, D = Q.shape
    Hk, Nk = K.shape[1:3]
    dev = Q.get_device()
    if check:
        if not Q.is_cuda:
            raise TypeError("Q must be a CUDA tensor")
        if D not in ROW_WIDTHS:
            raise ValueError(f"D is {D}, expected one of {ROW_WIDTHS}")
        if Hk == 0 or Hq % Hk:
            raise ValueError(f"{Hq} query heads are not a multiple of {Hk} key heads")
        q = check_rows("Q", Q, (B, Hq, Nq, D), dev)
        k = check_rows("K", K, (B, Hk, Nk, D), dev)
        v = check_rows("V", V, (B, Hk, Nk, D), dev)
        small = (0 if lengths is None else check_small("lengths", lengths, _i32, (B,), dev),
                 0 if q_lengths is None else check_small("q_lengths", q_lengths, _i32, (B,), dev),
                 0 if q_offsets is None else check_small("q_offsets", q_offsets, _i32, (B,), dev),
                 0 if documents is None else check_small("documents", documents, _i32, (B, Nk), dev),
                 0 if prefix is None else check_small("prefix", prefix, _i32, (B,), dev),
                 0 if slopes is None else check_small("slopes", slopes, _f32, (Hq,), dev))
        if prefix is not None and not causal:
            raise ValueError("prefix goes with causal=True")
    else:
        q, k, v = rows(Q), rows(K), rows(V)
        small = (ptr(lengths), ptr(q_lengths), ptr(q_offsets), ptr(documents), ptr(prefix), ptr(slopes))
    return (B, Hq, Hk, Nq, Nk, D, bool(causal), scale, cap, *q, *k, *v, *small), (B, Hq, Hk, Nq, Nk, D), dev


def _device_check(ws, stream, where):
    st = b.flare_last_device_status(ws, stream)
    if st != 0:
        raise b.FlareError(st, where + " (device status)")


def flare_attention_fwd(Q, K, V, lengths=None, q_lengths=None, q_offsets=None, documents=None, prefix=None,
                        slopes=None, causal: bool = False, scale: float = 0.0, cap: float = 0.0, Y=None, L_out=None,
                        workspace=None, stream=None, check: bool = True, device_check: bool = False):
    """Y = softmax(scores) V for Q [B,Hq,Nq,D], K, V [B,Hk,Nk,D] (bf16 views with
    dense rows; query head h reads key head h // (Hq // Hk)) -> Y [B,Hq,Nq,D] bf16.

    Row i stands at position p = q_offsets[b] + i (default Nk - Nq + i).  Scores:
    scale <q, k> (scale <= 0: 1/sqrt(D)), then cap * tanh(. / cap) if cap > 0,
    then minus slopes[h] * |p - j| (float32 [Hq]).  A row sees key j if j <
    lengths[b], i < q_lengths[b] (int32 [B]), with ``causal`` j <= p or j <
    prefix[b] (int32 [B]), and with ``documents`` (int32 [B,Nk]) j and p lie in
    the same run of equal ids >= 0.  A row that sees nothing comes out as zeros;
    keys that no row sees and rows behind q_lengths may hold anything.

    One new token over a cache: Nq = 1, lengths = tokens in the cache, q_offsets
    = lengths - 1.  ``L_out`` (float32 [B,Hq,Nq]) receives the rows'
    log-sum-exps.  With ``device_check`` the device status is read after the
    call (synchronises); its only error is an expired bounded wait."""
    head, sizes, dev = _head(Q, K, V, lengths, q_lengths, q_offsets, documents, prefix, slopes, causal, scale, cap,
                             check)
    Y, y = _output("Y", Y, Q, dev, stream, check)
    if L_out is None:
        L = 0
    else:
        L = check_small("L", L_out, _f32, Q.shape[:3], dev) if check else L_out.data_ptr()
    ws = _ws(workspace, flare_attention_workspace_bytes(*sizes), Q, stream)
    args = _ARGS.pack(*head, *y, L, *_NO_BACKWARD)
    call("flare_attention_fwd", "flare_attention_fwd", dev, stream, args, ws.data_ptr(), ws.numel())
    if device_check:
        _device_check(ws, stream, "flare_attention_fwd")
    return Y


def flare_attention_fwd_train(Q, K, V, lengths=None, q_lengths=None, q_offsets=None, documents=None, prefix=None,
                              slopes=None, causal: bool = False, scale: float = 0.0, cap: float = 0.0, Y=None,
                              L_out=None, workspace=None, stream=None, check: bool = True, device_check: bool = False):
    """flare_attention_fwd that returns (Y, L), what flare_attention_bwd takes."""
    if L_out is None:
        L_out = new(lambda: torch.empty(Q.shape[:3], dtype=_f32, device=Q.device), stream)
    Y = flare_attention_fwd(Q, K, V, lengths, q_lengths, q_offsets, documents, prefix, slopes, causal, scale, cap, Y,
                            L_out, workspace, stream, check, device_check)
    return Y, L_out


def flare_attention_bwd(Q, K, V, Y, L, dY, lengths=None, q_lengths=None, q_offsets=None, documents=None, prefix=None,
                        slopes=None, causal: bool = False, scale: float = 0.0, cap: float = 0.0, dQ=None, dK=None,
                        dV=None, workspace=None, stream=None, check: bool = True, device_check: bool = False):
    """Gradients (dQ, dK, dV), bf16, given dY and the forward's Y and L (same
    inputs, masks, scale and cap).  dK and dV are summed over the query heads of
    a key head.  dQ, dK and dV may be preallocated strided views."""
    head, sizes, dev = _head(Q, K, V, lengths, q_lengths, q_offsets, documents, prefix, slopes, causal, scale, cap,
                             check)
    if L is None:
        raise ValueError("L is the forward's log-sum-exps")
    if check:
        y, dy = check_rows("Y", Y, Q.shape, dev), check_rows("dY", dY, Q.shape, dev)
        check_small("L", L, _f32, Q.shape[:3], dev)
    else:
        y, dy = rows(Y), rows(dY)
    dQ, dq = _output("dQ", dQ, Q, dev, stream, check)
    dK, dk = _output("dK", dK, K, dev, stream, check)
    dV, dv = _output("dV", dV, K, dev, stream, check)
    ws = _ws(workspace, flare_attention_workspace_bytes(*sizes, backward=True), Q, stream)
    args = _ARGS.pack(*head, *y, L.data_ptr(), *dy, *dq, *dk, *dv)
    call("flare_attention_bwd", "flare_attention_bwd", dev, stream, args, ws.data_ptr(), ws.numel())
    if device_check:
        _device_check(ws, stream, "flare_attention_bwd")
    return dQ, dK, dV


class Attention(torch.autograd.Function):
    """Y of Q, K and V, differentiable in all three."""

    @staticmethod
    def forward(ctx, Q, K, V, lengths, q_lengths, q_offsets, documents, prefix, slopes, causal, scale, cap):
        Y, L = flare_attention_fwd_train(Q, K, V, lengths, q_lengths, q_offsets, documents, prefix, slopes, causal,
                                         scale, cap)
        ctx.save_for_backward(Q, K, V, Y, L, lengths, q_lengths, q_offsets, documents, prefix, slopes)
        ctx.causal, ctx.scale, ctx.cap = causal, scale, cap
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        Q, K, V, Y, L, *masks = ctx.saved_tensors
        dQ, dK, dV = flare_attention_bwd(Q, K, V, Y, L, dense(dY), *masks, ctx.causal, ctx.scale, ctx.cap)
        return (dQ, dK, dV) + (None,) * 9


def flare_attention(Q, K, V, lengths=None, q_lengths=None, q_offsets=None, documents=None, prefix=None, slopes=None,
                    causal: bool = False, scale: float = 0.0, cap: float = 0.0):
    """Differentiable flare_attention_fwd (see Attention)."""
    no_gradient("distance bias", slopes=slopes)
    return Attention.apply(Q, K, V, lengths, q_lengths, q_offsets, documents, prefix, slopes, causal, scale, cap)
