"""The preparation of queries and keys against its definition in 64 bits.

Tolerances.  An output is rounded to bf16 once: half a step is 2^-8 of the
value.  Before that everything is fp32 (2^-24 a step, `STEP`): the row's sum of
squares takes at most D roundings, the reciprocal root, the gain, cosine, sine
and the products a few more, fewer than 16 together, so each of the two terms
of a rotated value is off by at most (D + 16) steps of its magnitude.  The
backward has a second sum of D terms and as many products again; a gain's
gradient adds one rounding per summed row at worst.
"""
import math

import pytest
import torch

import rank_latent_routing_flare_b200 as fl

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP, HALF_BF16 = 2.0 ** -24, torch.finfo(torch.bfloat16).eps / 2


def packed_heads(B, N, H, D, g, layout):
    """[B, H, N, D] bf16 rows as a head-major tensor or a slice of a wider token-major one."""
    if layout == "head":
        return torch.randn(B, H, N, D, generator=g, device=DEV).bfloat16()
    wide = torch.randn(B, N, (H + 3) * D + 8, generator=g, device=DEV).bfloat16()
    return wide[:, :, 8 + D:8 + (H + 1) * D].unflatten(-1, (H, D)).transpose(1, 2)


def angles(N, freqs, positions, B):
    f = freqs.double().reshape(-1, freqs.shape[-1])
    if positions is None:
        pos = torch.arange(N, device=DEV).double().view(1, N, 1).expand(B, N, 1)
    else:
        pos = positions.double().reshape(B, N, -1)
    return pos @ f                                                  # [B, N, P]


def turn(v, a, interleaved):
    """(v turned by the angles a, the sum of the magnitudes of the terms of each element)."""
    P = a.shape[-1]
    R = 2 * P
    i, j = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, P), slice(P, R))
    c, s = a.cos().unsqueeze(1), a.sin().unsqueeze(1)
    out, mag = v.clone(), v.abs().clone()
    out[..., i], out[..., j] = v[..., i] * c - v[..., j] * s, v[..., i] * s + v[..., j] * c
    mag[..., i] = mag[..., j] = v[..., i].abs() + v[..., j].abs()
    return out, mag


def live(lengths, B, N):
    n = torch.full((B,), N, device=DEV) if lengths is None else lengths.clamp(0, N)
    return (torch.arange(N, device=DEV) < n.view(-1, 1)).view(B, 1, N, 1)


def reference(x, gain, a, lengths, eps, interleaved, dy=None):
    B, H, N, D = x.shape
    ok = live(lengths, B, N)
    x = torch.where(ok, x.double(), 0.0)
    g = torch.ones(H, 1, D, device=DEV, dtype=torch.float64) if gain is None else gain.double().expand(H, D).unsqueeze(1)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    y, mag = (x * r * g, (x * r * g).abs()) if a is None else turn(x * r * g, a, interleaved)
    if dy is None:
        y, mag = torch.where(ok, y, 0.0), torch.where(ok, mag, 0.0)
        return y, HALF_BF16 * y.abs() + (D + 16) * STEP * mag * (1 + HALF_BF16)
    dy = torch.where(ok, dy.double(), 0.0)
    u, umag = (dy, dy.abs()) if a is None else turn(dy, -a, interleaved)
    n = x * r
    w, wmag = u * g, umag * g.abs()
    dx = r * (w - n * (w * n).mean(-1, keepdim=True))
    dmag = r * (wmag + n.abs() * (wmag * n.abs()).mean(-1, keepdim=True))
    tol = HALF_BF16 * dx.abs() + (2 * D + 32) * STEP * dmag * (1 + HALF_BF16)
    dims = (0, 2) if gain is not None and gain.dim() == 2 else (0, 1, 2)
    dgain, gtol = (u * n).sum(dims), (umag * n.abs()).sum(dims) * (D + 32 + B * H * N) * STEP
    return torch.where(ok, dx, 0.0), torch.where(ok, tol, 0.0), dgain, gtol


def close(got, want, tol, what):
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    over = (got.double() - want).abs() - tol
    assert over.max() <= 0, (what, over.max().item())


def case(B, N, Hq, Hk, D, pos, gain, lengths, layout, rot, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    Q = packed_heads(B, N, Hq, D, g, layout) if Hq else None
    K = packed_heads(B, N, Hk, D, g, layout) if Hk else None
    gains = [None if gain == "none" or not H else 1 + 0.3 * torch.randn(*((H, D) if gain == "head" else (D,)),
                                                                      generator=g, device=DEV) for H in (Hq, Hk)]
    freqs = positions = None
    if rot:
        P = rot // 2
        if pos in ("none", "int"):
            freqs = (10000.0 ** (-torch.arange(P, device=DEV, dtype=torch.float64) / P)).float()
            if pos == "int":
                positions = torch.randint(-1000, 1 << 24, (B, N), generator=g, device=DEV, dtype=torch.int32)
        else:
            axes = int(pos[-1])
            freqs = 40 * torch.randn(axes, P, generator=g, device=DEV)
            positions = 2 * torch.rand(B, N, axes, generator=g, device=DEV) - 1
    n = None if lengths is None else torch.tensor([lengths[b % len(lengths)] for b in range(B)], dtype=torch.int32,
                                                  device=DEV)
    return Q, K, gains, freqs, positions, n, g


CASES = [
    # B, N, Hq, Hk, D, pos, gain, lengths, layout, rot, interleaved
    (1, 1, 1, 1, 16, "none", "none", None, "head", 16, False),
    (1, 1, 0, 3, 32, "int", "shared", None, "packed", 32, True),
    (3, 2, 5, 0, 64, "coord2", "head", (1, 0, 2), "packed", 32, False),
    (2, 3, 8, 2, 128, "int", "shared", (3, -7), "head", 128, False),
    (5, 33, 4, 4, 16, "coord3", "head", (40, 1, 32, 33, 0), "packed", 16, True),
    (2, 257, 6, 3, 32, "int", "head", None, "packed", 16, False),
    (4, 1000, 32, 8, 128, "int", "shared", (999, 1000, 17, 256), "packed", 128, True),
    (1, 5001, 7, 1, 64, "coord1", "none", (4999,), "packed", 48, False),
    (3, 700, 2, 2, 128, "coord4", "shared", None, "head", 96, False),
    (2, 130, 3, 9, 16, "none", "head", (129, 5), "packed", 10, True),
    (1, 4096, 16, 4, 64, "none", "shared", None, "packed", 0, False),
    (2, 20000, 8, 8, 16, "int", "shared", (20000, 12345), "packed", 16, False),
    (1, 1000, 200, 56, 128, "int", "head", None, "packed", 64, True),
]


@pytest.mark.parametrize("c", CASES, ids=[str(i) for i in range(len(CASES))])
def test_forward_and_backward(c):
    B, N, Hq, Hk, D, pos, gain, lengths, layout, rot, il = c
    Q, K, (gq, gk), freqs, positions, n, g = case(B, N, Hq, Hk, D, pos, gain, lengths, layout, rot, seed=N + D)
    dy = [None if x is None else torch.randn(x.shape, generator=g, device=DEV).bfloat16() for x in (Q, K)]
    if n is not None:   # padding may hold anything
        for x in (Q, K, *dy):
            if x is not None:
                x.masked_fill_(~live(n, B, N), math.nan)
    a = None if freqs is None else angles(N, freqs, positions, B)
    opts = dict(freqs=freqs, positions=positions, lengths=n, eps=1e-5, interleaved=il)
    out = fl.flare_qk_norm_rope_fwd(Q, K, gq, gk, **opts)
    grads = fl.flare_qk_norm_rope_bwd(Q, K, *dy, gq, gk, **opts)
    again = fl.flare_qk_norm_rope_bwd(Q, K, *dy, gq, gk, **opts)
    for x, gain_, y, d, key, gkey in ((Q, gq, out[0], dy[0], "dQ", "dq_gain"), (K, gk, out[1], dy[1], "dK", "dk_gain")):
        if x is None:
            assert y is None and grads[key] is None and grads[gkey] is None
            continue
        assert y.is_contiguous()
        close(y, *reference(x, gain_, a, n, 1e-5, il), key[1:])
        dx, tol, dgain, gtol = reference(x, gain_, a, n, 1e-5, il, dy=d)
        close(grads[key], dx, tol, key)
        assert torch.equal(grads[key], again[key])
        if gain_ is None:
            assert grads[gkey] is None
        else:
            close(grads[gkey], dgain, gtol, gkey)
            assert torch.equal(grads[gkey], again[gkey])


def test_gradient_against_differences():
    """<gradient, direction> against central differences of the 64-bit definition."""
    B, N, H, D = 2, 9, 3, 32
    Q, K, (gq, gk), freqs, positions, n, g = case(B, N, H, H, D, "coord2", "head", (9, 4), "head", 32, seed=1)
    dy = torch.randn(K.shape, generator=g, device=DEV).bfloat16()
    grads = fl.flare_qk_norm_rope_bwd(K=K, dKr=dy, k_gain=gk, freqs=freqs, positions=positions, lengths=n)
    a = angles(N, freqs, positions, B)
    f = lambda x, w: (reference(x, w, a, n, 1e-6, False)[0] * dy.double()).sum()   # noqa: E731
    h = 1e-5
    for name, base, run in (("dK", K.double(), lambda t: f(t, gk)), ("dk_gain", gk.double(), lambda t: f(K, t))):
        step = torch.randn(base.shape, generator=g, device=DEV, dtype=torch.float64)
        want = (run(base + h * step) - run(base - h * step)) / (2 * h)
        got = (grads[name].double() * step).sum()
        # the gradient's own rounding, half a bf16 step an element (fp32 for the gain), and h^2 of the differences
        tol = (grads[name].double().abs() * step.abs()).sum() * HALF_BF16 + 1e-6
        assert (got - want).abs() <= tol, (name, got.item(), want.item())


def test_strided_outputs_and_autograd():
    """Outputs and gradients written into slices of packed tensors leave the rest alone; autograd hands the same out."""
    B, N, Hq, Hk, D = 2, 77, 4, 2, 32
    Q, K, (gq, gk), freqs, positions, n, g = case(B, N, Hq, Hk, D, "int", "shared", (77, 30), "packed", 32, seed=2)
    opts = dict(freqs=freqs, positions=positions, lengths=n)
    Qr, Kr = fl.flare_qk_norm_rope_fwd(Q, K, gq, gk, **opts)
    wide = torch.full((B, N, (Hq + Hk + 1) * D), 7.0, dtype=torch.bfloat16, device=DEV)
    view = wide.unflatten(-1, (-1, D)).transpose(1, 2)
    got = fl.flare_qk_norm_rope_fwd(Q, K, gq, gk, Qr=view[:, :Hq], Kr=view[:, Hq + 1:], **opts)
    assert torch.equal(got[0], Qr) and torch.equal(got[1], Kr) and (view[:, Hq] == 7).all()
    dq, dk = torch.randn_like(Qr), torch.randn_like(Kr)
    want = fl.flare_qk_norm_rope_bwd(Q, K, dq, dk, gq, gk, **opts)
    wide.fill_(7.0)
    grads = fl.flare_qk_norm_rope_bwd(Q, K, dq, dk, gq, gk, grads={"dQ": view[:, :Hq], "dK": view[:, Hq + 1:]}, **opts)
    assert torch.equal(grads["dQ"], want["dQ"]) and (view[:, Hq] == 7).all()
    leaves = [t.detach().clone().requires_grad_() for t in (Q, K, gq, gk)]
    yq, yk = fl.flare_qk_norm_rope(*leaves, freqs, positions, n)
    torch.autograd.backward((yq, yk), (dq, dk))
    for leaf, key in zip(leaves, ("dQ", "dK", "dq_gain", "dk_gain")):
        assert torch.equal(leaf.grad, want[key]), key
    # only the keys' output is used, through an expanded gradient
    leaves = [t.detach().clone().requires_grad_() for t in (Q, K, gq, gk)]
    fl.flare_qk_norm_rope(*leaves, freqs, positions, n)[1].float().sum().backward()
    assert (leaves[0].grad == 0).all() and torch.isfinite(leaves[1].grad).all()
    with pytest.raises(ValueError):
        fl.flare_qk_norm_rope(*leaves, freqs.requires_grad_(), positions, n)


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart: the last heads and tokens of a large packed projection."""
    B, N, H, D = 1, (1 << 20) + 3, 2, 16
    wide = torch.empty(B, N, 2176, dtype=torch.bfloat16, device=DEV)
    K = wide[:, :, -H * D:].unflatten(-1, (H, D)).transpose(1, 2)
    g = torch.Generator(device=DEV).manual_seed(5)
    K.copy_(torch.randn(K.shape, generator=g, device=DEV))
    freqs = torch.rand(8, generator=g, device=DEV)
    _, Kr = fl.flare_qk_norm_rope_fwd(K=K, freqs=freqs)
    close(Kr, *reference(K, None, angles(N, freqs, None, B), None, 1e-6, False), "Kr")


def test_streams_and_graph():
    Q, K, (gq, gk), freqs, positions, n, g = case(2, 300, 4, 4, 64, "int", "shared", (300, 100), "packed", 64, seed=3)
    dq, dk = (torch.randn(x.shape, generator=g, device=DEV).bfloat16() for x in (Q, K))
    opts = dict(freqs=freqs, positions=positions, lengths=n)
    want = fl.flare_qk_norm_rope_fwd(Q, K, gq, gk, **opts)
    wgrad = fl.flare_qk_norm_rope_bwd(Q, K, dq, dk, gq, gk, **opts)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fl.flare_qk_norm_rope_fwd(Q, K, gq, gk, stream=side, **opts)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fl.flare_qk_norm_rope_fwd(Q, K, gq, gk, **opts)
        grads = fl.flare_qk_norm_rope_bwd(Q, K, dq, dk, gq, gk, **opts)
    saved = Q.clone()
    Q.mul_(3.0).add_(1.0)
    changed = fl.flare_qk_norm_rope_fwd(Q, K, gq, gk, **opts)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], changed[0]) and not torch.equal(out[0], want[0])
    Q.copy_(saved)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(grads["dq_gain"], wgrad["dq_gain"])


def test_python_refusals():
    x = torch.zeros(1, 2, 8, 32, dtype=torch.bfloat16, device=DEV)
    f = torch.zeros(16, device=DEV)
    for bad in (dict(Q=x.half()), dict(Q=x[..., :16].contiguous()[..., ::2]), dict(Q=x, K=x[:, :, :4]),
                dict(Q=x, freqs=f.double()), dict(Q=x, positions=torch.zeros(1, 8, device=DEV)),
                dict(Q=x, freqs=f, positions=torch.zeros(1, 7, device=DEV, dtype=torch.int32)),
                dict(Q=x, freqs=torch.zeros(2, 16, device=DEV)), dict(Q=x, q_gain=torch.ones(16, device=DEV)),
                dict(Q=x, k_gain=torch.ones(32, device=DEV)), dict(Q=x, lengths=torch.ones(2, device=DEV, dtype=torch.int32)),
                dict(Q=x, Qr=x[:, :1].expand(1, 2, 8, 32)), dict(Q=x, Kr=x), dict(Q=torch.zeros(1, 1, 2, 24, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            fl.flare_qk_norm_rope_fwd(**bad)
    with pytest.raises(fl.FlareError):
        fl.flare_qk_norm_rope_fwd(x, freqs=torch.zeros(20, device=DEV))   # rot = 40 > D
    with pytest.raises(ValueError):
        fl.flare_qk_norm_rope_bwd(Q=x)
