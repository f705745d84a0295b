"""Preparation of queries and keys: per-head RMS norm, gain and position
rotation in one pass, and its gradients.

A token projection gives queries and keys token-major; the mixer and the
attention take [B, H, N, D].  These calls read [B, H, N, D] views with any
strides (a slice of a packed projection, say) and write head-major tensors.
Argument checks and marshalling only: the kernels are behind
include/flare_ops.h.
"""
from __future__ import annotations

import struct

import torch

from . import _binding as b
from ._rows import ROW_WIDTHS, call, check_rows, check_small, ptr, rows, same_device, workspace as _ws

# flare_qk_norm_rope_args
_ARGS = struct.Struct("=9qd3q4q4q2q2q4q4q4q4q2q")


def flare_qk_norm_rope_workspace_bytes(B: int, N: int, Hq: int, Hk: int, D: int) -> int:
    return int(b.load_library().flare_qk_norm_rope_workspace_bytes(B, N, Hq, Hk, D))


def _sizes(Q, K, freqs, positions, lengths, q_gain, k_gain, check):
    X = Q if Q is not None else K
    if X is None:
        raise ValueError("Q and K are both None")
    if X.dim() != 4 or (K is not None and K.dim() != 4):
        raise ValueError("Q and K are [B, H, N, D]")
    B, _, N, D = X.shape
    Hq = 0 if Q is None else Q.shape[1]
    Hk = 0 if K is None else K.shape[1]
    rot, axes, kind = 0, 0, 0
    if freqs is not None:
        axes, rot = (1, 2 * freqs.shape[0]) if freqs.dim() == 1 else (freqs.shape[0], 2 * freqs.shape[-1])
        kind = 0 if positions is None else 1 if positions.dtype == torch.int32 else 2
    if check:
        dev = X.device
        if D not in ROW_WIDTHS:
            raise ValueError(f"D is {D}, expected one of {ROW_WIDTHS}")
        for name, t, H in (("Q", Q, Hq), ("K", K, Hk)):
            if t is not None:
                check_rows(name, t, (B, H, N, D))
        same_device(dev, Q=Q, K=K)
        for name, g, H in (("q_gain", q_gain, Hq), ("k_gain", k_gain, Hk)):
            if g is not None:
                if H == 0:
                    raise ValueError(f"{name} is given without its tensor")
                check_small(name, g, torch.float32, (D,) if g.dim() == 1 else (H, D), dev)
        if freqs is None:
            if positions is not None:
                raise ValueError("positions are given without freqs")
        else:
            if freqs.dim() not in (1, 2):
                raise ValueError("freqs is [rot / 2] or [axes, rot / 2]")
            check_small("freqs", freqs, torch.float32, None, dev)
            if kind == 1:
                check_small("positions", positions, torch.int32, (B, N), dev)
            elif kind == 2:
                shapes = ((B, N, axes), (B, N)) if axes == 1 else ((B, N, axes),)
                check_small("positions", positions, torch.float32,
                            positions.shape if tuple(positions.shape) in shapes else shapes[0], dev)
            if kind != 2 and axes != 1:
                raise ValueError("more than one axis of frequencies needs real coordinates (float32 positions)")
        check_small("lengths", lengths, torch.int32, (B,), dev)
    return B, N, D, Hq, Hk, rot, axes, kind, X.device


def _pack(sizes, interleaved, eps, freqs, positions, lengths, Q, K, q_gain, k_gain, Qr, Kr, dQ=None, dK=None,
          dq_gain=None, dk_gain=None):
    B, N, D, Hq, Hk, rot, axes, kind, _ = sizes
    return _ARGS.pack(B, N, D, Hq, Hk, rot, axes, bool(interleaved), kind, eps, ptr(freqs), ptr(positions),
                      ptr(lengths), *rows(Q), *rows(K), ptr(q_gain), ptr(k_gain),
                      q_gain is not None and q_gain.dim() == 2, k_gain is not None and k_gain.dim() == 2, *rows(Qr),
                      *rows(Kr), *rows(dQ), *rows(dK), ptr(dq_gain), ptr(dk_gain))


def _output(name, t, like, check):
    if like is None:
        if t is not None:
            raise ValueError(f"{name} is given without its input")
        return None
    if t is None:
        return torch.empty(like.shape, dtype=torch.bfloat16, device=like.device)
    if check:
        check_rows(name, t, tuple(like.shape), output=True)
        same_device(like.device, **{name: t})
    return t


def flare_qk_norm_rope_fwd(Q=None, K=None, q_gain=None, k_gain=None, freqs=None, positions=None, lengths=None,
                           eps: float = 1e-6, interleaved: bool = False, Qr=None, Kr=None, stream=None,
                           check: bool = True):
    """Per row x of Q [B,Hq,N,D] and K [B,Hk,N,D] (bf16 views with dense rows;
    either may be None): y = x * rsqrt(mean(x^2) + eps) * gain, then the pairs
    of y are rotated by the angles positions @ freqs.  Returns (Qr, Kr),
    head-major bf16 (or the given outputs).

    gains: float32 [D] or [H, D].  freqs: float32 [rot/2] or [axes, rot/2];
    None: no rotation.  positions: None (the token index), int32 [B, N], or
    float32 [B, N, axes] coordinates.  Pairs are (p, p + rot/2), with rot a
    multiple of 16, or (2p, 2p + 1) when ``interleaved``.  Rows n >=
    lengths[b] (int32 [B]) are not read and come out as zeros."""
    sizes = _sizes(Q, K, freqs, positions, lengths, q_gain, k_gain, check)
    Qr, Kr = _output("Qr", Qr, Q, check), _output("Kr", Kr, K, check)
    args = _pack(sizes, interleaved, eps, freqs, positions, lengths, Q, K, q_gain, k_gain, Qr, Kr)
    call(b.load_library().flare_qk_norm_rope_fwd, "flare_qk_norm_rope_fwd", sizes[-1], stream, args)
    return Qr, Kr


def flare_qk_norm_rope_bwd(Q=None, K=None, dQr=None, dKr=None, q_gain=None, k_gain=None, freqs=None, positions=None,
                           lengths=None, eps: float = 1e-6, interleaved: bool = False, grads=None, workspace=None,
                           stream=None, check: bool = True):
    """Gradients of flare_qk_norm_rope_fwd given those of its outputs.  Returns
    a dict: dQ, dK (bf16 [B,H,N,D]) and dq_gain, dk_gain (float32, the gains'
    shapes), None for what is absent.  ``grads`` may hold preallocated outputs
    by name; dQ and dK may be strided views (slices of a packed gradient)."""
    sizes = _sizes(Q, K, freqs, positions, lengths, q_gain, k_gain, check)
    B, N, D, Hq, Hk, _, _, _, dev = sizes
    for name, t, x in (("dQr", dQr, Q), ("dKr", dKr, K)):
        if (t is None) != (x is None):
            raise ValueError(f"{name} goes with its input")
        if check and t is not None:
            check_rows(name, t, tuple(x.shape))
            same_device(dev, **{name: t})
    g = dict(grads or {})
    g["dQ"], g["dK"] = _output("dQ", g.get("dQ"), Q, check), _output("dK", g.get("dK"), K, check)
    for name, gain in (("dq_gain", q_gain), ("dk_gain", k_gain)):
        if gain is None:
            g[name] = None
        elif g.get(name) is None:
            g[name] = torch.empty_like(gain)
        elif check:
            check_small(name, g[name], torch.float32, tuple(gain.shape), dev)
    ws = None
    if q_gain is not None or k_gain is not None:
        ws = _ws(workspace, flare_qk_norm_rope_workspace_bytes(B, N, Hq, Hk, D), dev)
    args = _pack(sizes, interleaved, eps, freqs, positions, lengths, Q, K, q_gain, k_gain, dQr, dKr, g["dQ"], g["dK"],
                 g["dq_gain"], g["dk_gain"])
    call(b.load_library().flare_qk_norm_rope_bwd, "flare_qk_norm_rope_bwd", dev, stream, args, ptr(ws),
         0 if ws is None else ws.numel())
    return g


class QkNormRope(torch.autograd.Function):
    """(Qr, Kr) of Q and K, differentiable in Q, K and the gains."""

    @staticmethod
    def forward(ctx, Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved):
        for name, t in (("freqs", freqs), ("positions", positions)):
            if t is not None and t.requires_grad:
                raise ValueError(f"{name}: gradients with respect to the angles are not computed")
        ctx.save_for_backward(Q, K, q_gain, k_gain, freqs, positions, lengths)
        ctx.eps, ctx.interleaved = eps, interleaved
        return flare_qk_norm_rope_fwd(Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved)

    @staticmethod
    def backward(ctx, dQr, dKr):
        Q, K, q_gain, k_gain, freqs, positions, lengths = ctx.saved_tensors
        g = flare_qk_norm_rope_bwd(Q, K, _dense(dQr, Q), _dense(dKr, K), q_gain, k_gain, freqs, positions, lengths,
                                   ctx.eps, ctx.interleaved)
        return g["dQ"], g["dK"], g["dq_gain"], g["dk_gain"], None, None, None, None, None


def _dense(dy, x):
    """A gradient as rows the kernels can read (autograd may hand over expanded or fp32 tensors)."""
    if x is None:
        return None
    if dy is None:
        return torch.zeros(x.shape, dtype=torch.bfloat16, device=x.device)
    return dy.to(torch.bfloat16).contiguous()


def flare_qk_norm_rope(Q=None, K=None, q_gain=None, k_gain=None, freqs=None, positions=None, lengths=None,
                       eps: float = 1e-6, interleaved: bool = False):
    """Differentiable flare_qk_norm_rope_fwd (see QkNormRope)."""
    return QkNormRope.apply(Q, K, q_gain, k_gain, freqs, positions, lengths, eps, interleaved)
