"""Exact softmax attention in 64 bits, its gradients, and bounds of what the
kernels' roundings can make of them.

Roundings counted (STEP = 2^-24, HALF = 2^-8, half a bf16 step): the fp32 dot
products of the scores (D + 8 steps of the sum of magnitudes) and the few
fp32 operations behind them move a score by at most `ds`; weights are
exponentials of scores (an absolute error of a score is a relative error of its
weight) rounded to bf16 where they enter a product, with an fp32 sum of up to
Nk terms; outputs are rounded to bf16 once.  The backward's delta takes the
rounded Y, its dS enters a product in bf16.  A weight below 2^-126, the smallest
normal fp32 number (TINY), may come out as zero: an absolute error of up to TINY
of each weight that a row sees.  Subnormal outputs are a multiple of 2^-133,
which is less than TINY.
"""
import math

import torch

STEP, HALF, TINY = 2.0 ** -24, torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float32).tiny


def visible(B, Nq, Nk, dev, lengths=None, q_lengths=None, q_offsets=None, documents=None, prefix=None, causal=False):
    """[B, Nq, Nk] of which keys a row sees, straight from the definition, and the rows' positions [B, Nq]."""
    i, j = torch.arange(Nq, device=dev), torch.arange(Nk, device=dev)
    off = torch.full((B,), Nk - Nq, device=dev) if q_offsets is None else q_offsets.long()
    p = off.view(B, 1) + i
    ok = torch.ones(B, Nq, Nk, dtype=torch.bool, device=dev)
    if lengths is not None:
        ok &= j < lengths.view(B, 1, 1)
    if q_lengths is not None:
        ok &= (i < q_lengths.view(B, 1)).unsqueeze(2)
    if causal:
        see = j <= p.unsqueeze(2)
        if prefix is not None:
            see = see | (j < prefix.view(B, 1, 1))
        ok &= see
    if documents is not None:
        for b in range(B):
            ids = documents[b].tolist()
            run, k = [], -1
            for n in range(Nk):
                if n == 0 or ids[n] != ids[n - 1]:
                    k += 1
                run.append(k if ids[n] >= 0 else -1)
            run = torch.tensor(run, device=dev)
            inside = (p[b] >= 0) & (p[b] < Nk)
            mine = torch.where(inside, run[p[b].clamp(0, Nk - 1)], -1)
            ok[b] &= (mine.view(Nq, 1) == run.view(1, Nk)) & (mine.view(Nq, 1) >= 0)
    return ok, p


def attention(Q, K, V, dY=None, slopes=None, scale=0.0, cap=0.0, **masks):
    """{name: (value, tolerance)} of Y and L, with dY also of dQ, dK, dV."""
    B, Hq, Nq, D = Q.shape
    Hk, Nk = K.shape[1:3]
    G = Hq // Hk
    scale = scale if scale > 0 else 1 / math.sqrt(D)
    ok, p = visible(B, Nq, Nk, Q.device, **masks)
    used_k, used_q = ok.any(1).view(B, 1, Nk, 1), ok.any(2).view(B, 1, Nq, 1)
    q = torch.where(used_q, Q.double(), 0.0).view(B, Hk, G, Nq, D)
    k = torch.where(used_k, K.double(), 0.0).unsqueeze(2)
    v = torch.where(used_k, V.double(), 0.0).unsqueeze(2)
    ok, some = ok.view(B, 1, 1, Nq, Nk), used_q.view(B, 1, 1, Nq, 1)
    s = scale * (q @ k.transpose(-1, -2))
    ds = (D + 8) * STEP * scale * (q.abs() @ k.abs().transpose(-1, -2))
    dx = torch.ones_like(s)
    ddx = torch.zeros_like(s)
    if cap > 0:
        t = torch.tanh(s / cap)
        s, dx = cap * t, 1 - t * t
        ds = ds + cap * 8 * STEP
        ddx = 16 * STEP + 2 * ds / cap
    if slopes is not None:
        dist = (p.unsqueeze(2) - torch.arange(Nk, device=Q.device)).abs().double()
        bias = slopes.double().view(1, Hk, G, 1, 1) * dist.view(B, 1, 1, Nq, Nk)
        near = torch.where(ok, bias, math.inf).amin(-1, keepdim=True).clamp(max=1e300)
        s = s - bias
        ds = ds + 8 * STEP * (bias - near).clamp(min=0)   # the part all keys share is exact, but for L itself
    ds = ds + 4 * STEP * s.abs().clamp(max=1e4)
    s = torch.where(ok, s, -math.inf)
    # weights that vanish do not matter: the bound of a row's scores weighs keys by e^(s - max + 8)
    top = torch.where(some, s.amax(-1, keepdim=True), 0.0)
    eps = torch.where(ok & (s > top - 100), ds, 0.0).amax(-1, keepdim=True) * 2 + 2.0 ** -21 + Nk * STEP
    L = torch.logsumexp(s, -1, keepdim=True)
    P = torch.exp(s - torch.where(some, L, 0.0))
    y = P @ v
    seen = TINY * ok.double()
    ytol = TINY + seen @ v.abs() + HALF * y.abs() + (HALF + 2 * eps) * (P @ v.abs()) * (1 + HALF)
    Lv = L.view(B, Hq, Nq)
    lt = torch.where(some, eps + 8 * STEP * (L.abs() + top.abs()), 0.0)
    if slopes is not None:
        lt = lt + torch.where(some, 4 * STEP * near, 0.0)
    out = {"Y": (y.view(B, Hq, Nq, D), ytol.view(B, Hq, Nq, D)), "L": (Lv, lt.view(B, Hq, Nq))}
    if dY is None:
        return out
    dy = torch.where(used_q, dY.double(), 0.0).view(B, Hk, G, Nq, D)
    e1 = 2 * eps + lt                                                   # relative error of a recomputed weight
    g, delta = dy @ v.transpose(-1, -2), (dy * y).sum(-1, keepdim=True)
    dS = P * (g - delta) * dx
    gerr = (D + 8) * STEP * (dy.abs() @ v.abs().transpose(-1, -2))
    derr = (dy.abs() * (ytol + (D + 8) * STEP * y.abs())).sum(-1, keepdim=True)
    E = P * (((g - delta).abs() * (HALF + e1) + gerr + derr) * dx + (g - delta).abs() * ddx) * (1 + HALF)
    E = E + seen * (g - delta).abs()
    dq = scale * (dS @ k)
    dqt = TINY + HALF * dq.abs() + scale * ((E + Nk * STEP * dS.abs()) @ k.abs()) * (1 + HALF)
    n = G * Nq * STEP
    dk = scale * (dS.transpose(-1, -2) @ q).sum(2)
    dkt = TINY + HALF * dk.abs() + scale * ((E + n * dS.abs()).transpose(-1, -2) @ q.abs()).sum(2) * (1 + HALF)
    dv = (P.transpose(-1, -2) @ dy).sum(2)
    dvt = TINY + HALF * dv.abs() + ((P * (HALF + e1 + n) + seen).transpose(-1, -2) @ dy.abs()).sum(2) * (1 + HALF)
    out.update(dQ=(dq.view(B, Hq, Nq, D), dqt.view(B, Hq, Nq, D)), dK=(dk, dkt), dV=(dv, dvt))
    return out


def close(got, want, what):
    value, tol = want
    assert got.shape == value.shape, what
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(value)), what
    same = torch.where(torch.isfinite(value), (got - value).abs() - tol, torch.where(got == value, -1.0, 1.0))
    assert same.max() <= 0, (what, same.max().item(), int((same > 0).sum()), (same > 0).nonzero()[:4].tolist())
