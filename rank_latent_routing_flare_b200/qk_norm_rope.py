"""Preparation of queries and keys: per-head RMS norm, gain and position
rotation in one pass, and its gradients.

A token projection gives queries and keys token-major; the mixer and the
attention take [B, H, N, D].  These calls read [B, H, N, D] views with any
strides (a slice of a packed projection, say) and write head-major tensors.
Argument checks and marshalling only: the kernels are behind
include/flare_ops.h.
"""
from __future__ import annotations

import functools
import struct

import torch
from torch.autograd.function import once_differentiable

from ._rows import (NO_ROWS, ROW_WIDTHS, call, check_rows, check_small, dense, entry, new_like, no_gradient,
                    output as _output, ptr, rows, workspace as _ws)

# flare_qk_norm_rope_args
_ARGS = struct.Struct("=9qd3q4q4q2q2q4q4q4q4q2q")
_f32, _i32 = torch.float32, torch.int32
_NO_BACKWARD = NO_ROWS * 2 + (0, 0)


@functools.lru_cache(maxsize=4096)
def flare_qk_norm_rope_workspace_bytes(B: int, N: int, Hq: int, Hk: int, D: int) -> int:
    return int(entry("flare_qk_norm_rope_workspace_bytes")(B, N, Hq, Hk, D))


def _check_gain(name, g, H, D, dev):
    if H == 0:
        raise ValueError(f"{name} is given without its tensor")
    return _aligned(name, check_small(name, g, _f32, (D,) if g.dim() == 1 else (H, D), dev))


def _aligned(name, p):
    if p & 15:
        raise ValueError(f"{name} must lie on a 16-byte boundary")
    return p


def _head(Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved, check):
    """The inputs' part of the argument struct, in its order, and (B, N, D, Hq, Hk, device index)."""
    X = Q if Q is not None else K
    if X is None:
        raise ValueError("Q and K are both None")
    if X.dim() != 4 or (K is not None and K.dim() != 4):
        raise ValueError("Q and K are [B, H, N, D]")
    B, H, N, D = X.shape
    Hq = 0 if Q is None else H
    Hk = 0 if K is None else K.shape[1]
    rot = axes = kind = 0
    if freqs is not None:
        f = freqs.shape
        axes, rot = (1, 2 * f[0]) if len(f) == 1 else (f[0], 2 * f[-1])
        kind = 0 if positions is None else 1 if positions.dtype is _i32 else 2
    dev = X.get_device()
    if check:
        if not X.is_cuda:
            raise TypeError("Q and K must be CUDA tensors")
        if D not in ROW_WIDTHS:
            raise ValueError(f"D is {D}, expected one of {ROW_WIDTHS}")
        q = NO_ROWS if Q is None else check_rows("Q", Q, (B, Hq, N, D), dev)
        k = NO_ROWS if K is None else check_rows("K", K, (B, Hk, N, D), dev)
        gq = 0 if q_gain is None else _check_gain("q_gain", q_gain, Hq, D, dev)
        gk = 0 if k_gain is None else _check_gain("k_gain", k_gain, Hk, D, dev)
        fp = 0 if freqs is None else check_small("freqs", freqs, _f32, None, dev)
        n = 0 if lengths is None else check_small("lengths", lengths, _i32, (B,), dev)
        pp = 0
        if freqs is None:
            if positions is not None:
                raise ValueError("positions are given without freqs")
        else:
            if len(f) not in (1, 2):
                raise ValueError("freqs is [rot / 2] or [axes, rot / 2]")
            if kind == 1:
                pp = check_small("positions", positions, _i32, (B, N), dev)
            elif kind == 2:
                pp = check_small("positions", positions, _f32,
                                 (B, N) if axes == 1 and positions.dim() == 2 else (B, N, axes), dev)
            if kind != 2 and axes != 1:
                raise ValueError("more than one axis of frequencies needs real coordinates (float32 positions)")
    else:
        q, k = (NO_ROWS if t is None else rows(t) for t in (Q, K))
        gq, gk, fp, pp, n = ptr(q_gain), ptr(k_gain), ptr(freqs), ptr(positions), ptr(lengths)
    packed = (B, N, D, Hq, Hk, rot, axes, bool(interleaved), kind, eps, fp, pp, n, *q, *k, gq, gk,
              gq != 0 and q_gain.dim() == 2, gk != 0 and k_gain.dim() == 2)
    return packed, (B, N, D, Hq, Hk, dev)


def _side(name, t, like, dev, stream, check):
    """The output that goes with an input, which may be absent."""
    if like is not None:
        return _output(name, t, like, dev, stream, check)
    if t is not None:
        raise ValueError(f"{name} is given without its input")
    return None, NO_ROWS


def flare_qk_norm_rope_fwd(Q=None, K=None, q_gain=None, k_gain=None, freqs=None, positions=None, lengths=None,
                           eps: float = 1e-6, interleaved: bool = False, Qr=None, Kr=None, stream=None,
                           check: bool = True):
    """Per row x of Q [B,Hq,N,D] and K [B,Hk,N,D] (bf16 views with dense rows;
    either may be None): y = x * rsqrt(mean(x^2) + eps) * gain, then the pairs
    of y are rotated by the angles positions @ freqs.  Returns (Qr, Kr),
    head-major bf16 (or the given outputs).

    gains: float32 [D] or [H, D], on a 16-byte boundary.  freqs: float32
    [rot/2] or [axes, rot/2]; None: no rotation.  positions: None (the token
    index), int32 [B, N], or float32 [B, N, axes] coordinates.  Pairs are (p, p +
    rot/2), with rot a multiple of 16, or (2p, 2p + 1) when ``interleaved``.
    Rows n >= lengths[b] (int32 [B]) are not read and come out as zeros."""
    head, (*_, dev) = _head(Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved, check)
    Qr, q = _side("Qr", Qr, Q, dev, stream, check)
    Kr, k = _side("Kr", Kr, K, dev, stream, check)
    args = _ARGS.pack(*head, *q, *k, *_NO_BACKWARD)
    call("flare_qk_norm_rope_fwd", "flare_qk_norm_rope_fwd", dev, stream, args)
    return Qr, Kr


def flare_qk_norm_rope_bwd(Q=None, K=None, dQr=None, dKr=None, q_gain=None, k_gain=None, freqs=None, positions=None,
                           lengths=None, eps: float = 1e-6, interleaved: bool = False, grads=None, workspace=None,
                           stream=None, check: bool = True):
    """Gradients of flare_qk_norm_rope_fwd given those of its outputs.  Returns
    a dict: dQ, dK (bf16 [B,H,N,D]) and dq_gain, dk_gain (float32, the gains'
    shapes), None for what is absent.  ``grads`` may hold preallocated outputs
    by name; dQ and dK may be strided views (slices of a packed gradient)."""
    head, (B, N, D, Hq, Hk, dev) = _head(Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved, check)
    dy = []
    for name, t, x in (("dQr", dQr, Q), ("dKr", dKr, K)):
        if (t is None) != (x is None):
            raise ValueError(f"{name} goes with its input")
        dy += NO_ROWS if t is None else check_rows(name, t, x.shape, dev) if check else rows(t)
    g = dict(grads or {})
    g["dQ"], q = _side("dQ", g.get("dQ"), Q, dev, stream, check)
    g["dK"], k = _side("dK", g.get("dK"), K, dev, stream, check)
    for name, gain in (("dq_gain", q_gain), ("dk_gain", k_gain)):
        if gain is None:
            g[name] = None
        elif g.get(name) is None:
            g[name] = new_like(gain, stream)
        elif check:
            _aligned(name, check_small(name, g[name], _f32, gain.shape, dev))
    ws, nbytes = 0, 0
    if q_gain is not None or k_gain is not None:
        workspace = _ws(workspace, flare_qk_norm_rope_workspace_bytes(B, N, Hq, Hk, D), Q if Q is not None else K,
                        stream)
        ws, nbytes = workspace.data_ptr(), workspace.numel()
    args = _ARGS.pack(*head, *dy, *q, *k, ptr(g["dq_gain"]), ptr(g["dk_gain"]))
    call("flare_qk_norm_rope_bwd", "flare_qk_norm_rope_bwd", dev, stream, args, ws, nbytes)
    return g


class QkNormRope(torch.autograd.Function):
    """(Qr, Kr) of Q and K, differentiable in Q, K and the gains."""

    @staticmethod
    def forward(ctx, Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved):
        ctx.save_for_backward(Q, K, q_gain, k_gain, freqs, positions, lengths)
        ctx.eps, ctx.interleaved = eps, interleaved
        return flare_qk_norm_rope_fwd(Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dQr, dKr):
        Q, K, q_gain, k_gain, freqs, positions, lengths = ctx.saved_tensors
        g = flare_qk_norm_rope_bwd(Q, K, _dense(dQr, Q), _dense(dKr, K), q_gain, k_gain, freqs, positions, lengths,
                                   ctx.eps, ctx.interleaved)
        return g["dQ"], g["dK"], g["dq_gain"], g["dk_gain"], None, None, None, None, None


def _dense(dy, x):
    if x is None:
        return None
    if dy is None:
        return torch.zeros(x.shape, dtype=torch.bfloat16, device=x.device)
    return dense(dy)


def flare_qk_norm_rope(Q=None, K=None, q_gain=None, k_gain=None, freqs=None, positions=None, lengths=None,
                       eps: float = 1e-6, interleaved: bool = False):
    """Differentiable flare_qk_norm_rope_fwd (see QkNormRope)."""
    no_gradient("angles", freqs=freqs, positions=positions)
    return QkNormRope.apply(Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved)
