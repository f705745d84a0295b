"""Exact softmax attention, forward and backward, against its definition in 64
bits (attention_ref holds the tolerances and their derivation)."""
import math

import pytest
import torch

import rank_latent_routing_flare_b200 as fl

from . import attention_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def heads(B, H, N, D, g, layout, scale=1.0):
    x = scale * torch.randn(B, N, H + 1, D, generator=g, device=DEV)
    if layout == "head":
        return x[:, :, :H].transpose(1, 2).bfloat16().contiguous()
    return x.bfloat16()[:, :, 1:].transpose(1, 2)        # a slice of a token-major projection


def documents(B, N, cuts, dead=()):
    """Ids of runs that begin at `cuts`; positions of the runs listed in `dead` get id -1."""
    ids = torch.zeros(N, dtype=torch.int32)
    for n, c in enumerate(cuts):
        ids[c:] = -1 if n + 1 in dead else 10 - n
    return ids.expand(B, N).contiguous().to(DEV)


def make(B, Hq, Hk, Nq, Nk, D, seed, layout="packed", qscale=1.5, **opts):
    g = torch.Generator(device=DEV).manual_seed(seed)
    Q, K, V = heads(B, Hq, Nq, D, g, layout, qscale), heads(B, Hk, Nk, D, g, layout), heads(B, Hk, Nk, D, g, layout)
    dY = torch.randn(B, Hq, Nq, D, generator=g, device=DEV).bfloat16()
    if opts.pop("bias", False):
        opts["slopes"] = 2.0 ** -torch.linspace(1, 8, Hq, device=DEV)
    return Q, K, V, dY, opts


def poison(Q, K, V, dY, opts):
    """NaN and infinities wherever nothing may be read."""
    masks = {n: opts.get(n) for n in ("lengths", "q_lengths", "q_offsets", "documents", "prefix", "causal")}
    masks["causal"] = bool(masks["causal"])
    B, _, Nq, _ = Q.shape
    Nk = K.shape[2]
    dead_k, dead_q = torch.zeros(B, Nk, dtype=torch.bool, device=DEV), torch.zeros(B, Nq, dtype=torch.bool, device=DEV)
    if opts.get("lengths") is not None:
        dead_k |= torch.arange(Nk, device=DEV) >= opts["lengths"].view(B, 1)
    if opts.get("documents") is not None:
        dead_k |= opts["documents"] < 0
        if Nq == Nk:
            dead_q |= opts["documents"] < 0
    if opts.get("q_lengths") is not None:
        dead_q |= torch.arange(Nq, device=DEV) >= opts["q_lengths"].view(B, 1)
    for x, m, bad in ((Q, dead_q, math.nan), (dY, dead_q, math.inf), (K, dead_k, math.nan), (V, dead_k, -math.inf)):
        x.masked_fill_(m.view(B, 1, -1, 1), bad)


def check(Q, K, V, dY, opts, backward=True):
    poison(Q, K, V, dY, opts)
    want = ref.attention(Q, K, V, dY=dY if backward else None, **opts)
    Y, L = fl.flare_attention_fwd_train(Q, K, V, device_check=True, **opts)
    ref.close(Y, want["Y"], "Y")
    ref.close(L, want["L"], "L")
    if not backward:
        return
    dQ, dK, dV = fl.flare_attention_bwd(Q, K, V, Y, L, dY, device_check=True, **opts)
    for name, got in (("dV", dV), ("dQ", dQ), ("dK", dK)):
        ref.close(got, want[name], name)
    again = fl.flare_attention_bwd(Q, K, V, Y, L, dY, **opts)
    assert all(torch.equal(x, y) for x, y in zip((dQ, dK, dV), again))


# B, Hq, Hk, Nq, Nk, options
SHAPES = {
    "one": (1, 1, 1, 1, 1, {}),
    "tiny": (2, 2, 1, 3, 5, {}),
    "rows17": (1, 1, 1, 17, 40, {"causal": True}),
    "square": (1, 2, 2, 128, 128, {"causal": True}),
    "odd": (2, 4, 2, 257, 257, {"causal": True, "bias": True}),
    "ragged": (3, 2, 1, 300, 300, {"lengths": (300, 1, 129), "q_lengths": (300, 1, 129)}),
    "empty": (3, 2, 2, 70, 70, {"lengths": (0, 70, 64), "q_lengths": (70, 0, 64), "cap": 5.0}),
    "out_of_range_lengths": (2, 1, 1, 50, 60, {"lengths": (-4, 99), "q_lengths": (60, 1000)}),
    "docs": (2, 4, 1, 500, 500, {"documents": ((70, 71, 200, 333), ()), "causal": True, "cap": 4.0}),
    "docs_dead": (1, 2, 2, 400, 400, {"documents": ((100, 190, 260), (2,)), "bias": True}),
    "docs_dead_tail": (2, 2, 1, 333, 333, {"documents": ((64, 200), (2,)), "causal": True}),
    "prefix": (2, 2, 1, 391, 391, {"causal": True, "prefix": (0, 200)}),
    "prefix_long": (2, 1, 1, 150, 200, {"causal": True, "prefix": (500, -3), "bias": True}),
    "cross": (2, 4, 4, 130, 1000, {"lengths": (1000, 77), "cap": 10.0}),
    "latents": (1, 2, 2, 600, 90, {}),
    "before": (1, 2, 1, 200, 100, {"causal": True}),                       # rows 0 .. 99 stand before every key
    "offsets": (3, 2, 1, 64, 256, {"causal": True, "q_offsets": (0, 100, -70), "bias": True}),
    "offset_docs": (3, 2, 1, 64, 256, {"documents": ((90, 130), ()), "q_offsets": (60, -30, 230)}),
    "far": (2, 2, 1, 40, 200, {"q_offsets": (1 << 30, -(1 << 30)), "bias": True}),
    "long": (1, 2, 1, 1100, 1100, {"causal": True, "cap": 30.0, "bias": True}),
    "few_long": (1, 1, 1, 33, 5000, {}),                                   # split along the keys
    "few_long_causal": (2, 2, 1, 64, 3001, {"causal": True, "bias": True, "cap": 20.0, "lengths": (3001, 1500),
                                            "q_offsets": (2937, 1436)}),
}


def options(o, B, Nk):
    o = dict(o)
    for n in ("lengths", "q_lengths", "prefix", "q_offsets"):
        if n in o:
            o[n] = i32(*o[n])
    if "documents" in o:
        o["documents"] = documents(B, Nk, *o["documents"])
    return o


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("name", SHAPES)
def test_against_definition(name, D):
    B, Hq, Hk, Nq, Nk, o = SHAPES[name]
    check(*make(B, Hq, Hk, Nq, Nk, D, seed=D + Nq, layout="head" if D == 64 else "packed", **options(o, B, Nk)))


# Backward where CTAs share a key tile's rows (few key heads, many rows), where none does, and either side of the
# number of keys up to which the dQ pass sums twice.
BACKWARD = {
    "one_key_head": (1, 8, 1, 700, 300, {"cap": 9.0}),
    "one_key_head_causal": (1, 6, 1, 1300, 1300, {"causal": True, "documents": ((500, 777), ())}),
    "latents_ragged": (2, 2, 2, 3000, 40, {"lengths": (40, 17), "q_lengths": (2999, 3), "bias": True}),
    "one_batch_idle": (3, 2, 1, 600, 70, {"q_lengths": (600, 0, 0), "lengths": (70, 70, 0)}),
    "many_heads": (2, 16, 8, 300, 1300, {"lengths": (1300, 1111), "bias": True}),
    "keys_1024": (1, 3, 1, 200, 1024, {"causal": True, "q_offsets": (824,)}),
    "keys_1025": (1, 3, 1, 200, 1025, {"causal": True, "q_offsets": (824,)}),
}


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("name", BACKWARD)
def test_backward_shapes(name, D):
    B, Hq, Hk, Nq, Nk, o = BACKWARD[name]
    check(*make(B, Hq, Hk, Nq, Nk, D, seed=D + Nk, **options(o, B, Nk)))


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("G,Nq", [(1, 1), (4, 1), (3, 5), (16, 1), (1, 16), (2, 3)])
@pytest.mark.parametrize("Nk", [1, 15, 16, 700, 5003])
def test_few_rows(D, G, Nq, Nk):
    """Single tokens and a few rows over a cache: ragged lengths, the new tokens last, cap and bias."""
    B, Hk = 3, 2
    n = i32(Nk, max(1, Nk // 3), max(0, Nk - 1))
    opts = {"lengths": n, "q_offsets": n - Nq, "causal": True}
    if (D + Nk + G) % 3 == 0:
        opts.update(cap=8.0, bias=True)
    check(*make(B, Hk * G, Hk, Nq, Nk, D, seed=Nk + G, layout="head" if G == 4 else "packed", **opts), backward=False)


def test_few_rows_with_documents_and_prefix():
    opts = {"documents": documents(2, 900, (300, 450, 460), (2,)), "q_offsets": i32(448, 290)}
    check(*make(2, 4, 2, 8, 900, 64, seed=1, **opts), backward=False)
    opts = {"causal": True, "prefix": i32(700, 3), "q_offsets": i32(100, 0)}
    check(*make(2, 4, 2, 4, 900, 32, seed=2, **opts), backward=False)


def test_large_scores_and_growing_maxima():
    """Scores in the hundreds, whose running maximum grows in every tile, and identical keys."""
    for D in (16, 64, 128):
        Q, K, V, dY, _ = make(1, 2, 1, 260, 900, D, seed=3, qscale=8.0)
        K.mul_(torch.linspace(0.1, 6.0, 900, device=DEV).view(1, 1, -1, 1))
        check(Q, K, V, dY, {})
        check(Q, K, V, dY, {"cap": 15.0})
        K.copy_(K[:, :, :1].expand_as(K).clone())
        check(Q, K, V, dY, {"scale": 0.01})


@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("opts", [{}, {"cap": 20.0}, {"steep": True, "causal": True}, {"steep": True, "cap": 20.0}],
                         ids=["plain", "cap", "bias", "bias_cap"])
def test_nan_of_a_visible_key_shows(D, opts):
    """A NaN in a key or value that a row sees reaches the row, however small its weight would be."""
    opts = dict(opts)
    if opts.pop("steep", False):
        opts["slopes"] = torch.full((2,), 4.0, device=DEV)
    Q, K, V, _, _ = make(1, 2, 2, 700, 700, D, seed=11)
    for x in (K, V):
        old = x[0, 1, 3].clone()
        x[0, 1, 3] = math.nan
        Y = fl.flare_attention_fwd(Q, K, V, **opts)
        first = 3 if opts.get("causal") else 0
        assert torch.isnan(Y[0, 1, first:]).all() and torch.isfinite(Y[0, 0]).all()
        step = fl.flare_attention_fwd(Q[:, :, -1:], K, V, **opts)
        assert torch.isnan(step[0, 1]).all() and torch.isfinite(step[0, 0]).all()
        x[0, 1, 3] = old


def test_strided_outputs_streams_and_graph():
    Q, K, V, dY, o = make(2, 4, 2, 200, 200, 64, seed=4, causal=True, cap=10.0, documents=documents(2, 200, (90,)))
    Y, L = fl.flare_attention_fwd_train(Q, K, V, **o)
    g = fl.flare_attention_bwd(Q, K, V, Y, L, dY, **o)
    wide = torch.full((2, 200, 9, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    view = wide.transpose(1, 2)
    fl.flare_attention_fwd(Q, K, V, Y=view[:, :4], **o)
    assert torch.equal(view[:, :4], Y) and (view[:, 4:] == 7).all()
    fl.flare_attention_bwd(Q, K, V, view[:, :4].contiguous(), L, dY, dQ=view[:, :4], dK=view[:, 4:6], dV=view[:, 6:8], **o)
    assert torch.equal(view[:, :4], g[0]) and torch.equal(view[:, 4:6], g[1]) and torch.equal(view[:, 6:8], g[2])
    assert (view[:, 8] == 7).all()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    Y2 = fl.flare_attention_fwd(Q, K, V, stream=side, **o)
    side.synchronize()
    assert torch.equal(Y2, Y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Yg, Lg = fl.flare_attention_fwd_train(Q, K, V, **o)
        gg = fl.flare_attention_bwd(Q, K, V, Yg, Lg, dY, **o)
    K.mul_(0.5)
    o["documents"].copy_(documents(2, 200, (120, 150)))
    want, Lw = fl.flare_attention_fwd_train(Q, K, V, **o)
    wg = fl.flare_attention_bwd(Q, K, V, want, Lw, dY, **o)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Yg, want) and torch.equal(Lg, Lw) and not torch.equal(Yg, Y)
    assert all(torch.equal(x, y) for x, y in zip(gg, wg))


def test_step_matches_the_last_row():
    """A new token's row is the last row of the whole sequence, to the roundings of both."""
    Q, K, V, _, _ = make(2, 4, 2, 300, 300, 32, seed=5)
    slopes = 2.0 ** -torch.linspace(1, 8, 4, device=DEV)
    whole = fl.flare_attention_fwd(Q, K, V, causal=True, slopes=slopes)
    step = fl.flare_attention_fwd(Q[:, :, -1:], K, V, causal=True, slopes=slopes)
    want = ref.attention(Q[:, :, -1:], K, V, causal=True, slopes=slopes)["Y"]
    ref.close(step, want, "step")
    ref.close(whole[:, :, -1:], want, "whole")


def test_gradients_against_differences():
    Q, K, V, dY, o = make(1, 4, 2, 70, 70, 32, seed=6, layout="head", causal=True, cap=3.0, bias=True,
                          prefix=i32(20))
    Y, L = fl.flare_attention_fwd_train(Q, K, V, **o)
    grads = fl.flare_attention_bwd(Q, K, V, Y, L, dY, **o)
    g = torch.Generator(device=DEV).manual_seed(7)
    want = ref.attention(Q, K, V, dY=dY, **o)
    for n, key in enumerate(("dQ", "dK", "dV")):
        ts = [Q.double(), K.double(), V.double()]
        step = torch.randn(ts[n].shape, generator=g, device=DEV, dtype=torch.float64)
        up, down = list(ts), list(ts)
        up[n], down[n] = ts[n] + 1e-5 * step, ts[n] - 1e-5 * step
        f = lambda t: (ref.attention(*t, **o)["Y"][0] * dY.double()).sum()   # noqa: E731
        diff = (f(up) - f(down)) / 2e-5
        tol = (want[key][1] * step.abs()).sum() + 1e-6
        assert ((grads[n].double() * step).sum() - diff).abs() <= tol


def test_autograd():
    Q, K, V, dY, o = make(2, 4, 2, 90, 90, 64, seed=8, causal=True, lengths=i32(90, 40), q_lengths=i32(90, 40))
    Y, L = fl.flare_attention_fwd_train(Q, K, V, **o)
    g = fl.flare_attention_bwd(Q, K, V, Y, L, dY, **o)
    leaves = [t.detach().clone().requires_grad_() for t in (Q, K, V)]
    out = fl.flare_attention(*leaves, **o)
    assert torch.equal(out, Y)
    out.backward(dY)
    assert all(torch.equal(x.grad, y) for x, y in zip(leaves, g))
    with pytest.raises(ValueError):
        fl.flare_attention(*leaves, slopes=torch.ones(4, device=DEV, requires_grad=True))


def test_preparation_and_attention_together():
    """A projection's slices through the preparation and the attention and back: every gradient lands in the slice of
    one packed gradient, and matches 64-bit autograd to the roundings of the rows between the operators."""
    B, N, Hq, Hk, D = 2, 333, 4, 2, 32
    g = torch.Generator(device=DEV).manual_seed(9)
    packed = torch.randn(B, N, (Hq + 2 * Hk) * D, generator=g, device=DEV).bfloat16()
    rows = packed.unflatten(-1, (-1, D)).transpose(1, 2)
    Q, K, V = rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:]
    gains = [1 + 0.2 * torch.randn(D, generator=g, device=DEV) for _ in range(2)]
    freqs = 10000.0 ** (-torch.arange(D // 2, device=DEV) / (D // 2))
    n = i32(N, 200)
    Qr, Kr = fl.flare_qk_norm_rope_fwd(Q, K, *gains, freqs=freqs, lengths=n)
    masks = dict(causal=True, lengths=n, q_lengths=n)
    Y, L = fl.flare_attention_fwd_train(Qr, Kr, V, **masks)
    dY = torch.randn(Y.shape, generator=g, device=DEV).bfloat16()
    grad = torch.full_like(packed, 5.0)
    view = grad.unflatten(-1, (-1, D)).transpose(1, 2)
    dQr, dKr, _ = fl.flare_attention_bwd(Qr, Kr, V, Y, L, dY, dV=view[:, Hq + Hk:], **masks)
    out = fl.flare_qk_norm_rope_bwd(Q, K, dQr, dKr, *gains, freqs=freqs, lengths=n,
                                    grads={"dQ": view[:, :Hq], "dK": view[:, Hq:Hq + Hk]})
    # each operator against 64 bits on the rows that it was given
    want = ref.attention(Qr, Kr, V, dY=dY, **masks)
    ref.close(Y, want["Y"], "Y")
    ref.close(view[:, Hq + Hk:], want["dV"], "dV")
    ref.close(dQr, want["dQ"], "dQr")
    from .test_gpu_qk_norm_rope import angles, close, reference
    a = angles(N, freqs, None, B)
    for x, gain, d, key in ((Q, gains[0], dQr, "dQ"), (K, gains[1], dKr, "dK")):
        dx, tol, dgain, gtol = reference(x, gain, a, n, 1e-6, False, dy=d)
        close(out[key], dx, tol, key)
        close(out["d" + key[1].lower() + "_gain"], dgain, gtol, key)
    assert (grad[1, 200:] == 0).all() and torch.isfinite(grad).all()


def test_prepared_keys_feed_the_mixer():
    """The mixer takes prepared keys as they come out: same layout, same result as on a copy."""
    B, N, H, D, M = 2, 500, 4, 16, 32
    g = torch.Generator(device=DEV).manual_seed(10)
    packed = torch.randn(B, N, 2 * H * D, generator=g, device=DEV).bfloat16()
    rows = packed.unflatten(-1, (-1, D)).transpose(1, 2)
    coords = torch.rand(B, N, 3, generator=g, device=DEV)
    _, Kr = fl.flare_qk_norm_rope_fwd(K=rows[:, :H], freqs=3 * torch.randn(3, D // 2, generator=g, device=DEV),
                                      positions=coords)
    Q = torch.randn(H, M, D, generator=g, device=DEV).bfloat16()
    V = rows[:, H:].contiguous()
    Y = fl.flare_mixer_fwd(Kr, V, Q)
    k, v, q = Kr.double(), V.double(), Q.double()
    z = torch.softmax(q @ k.transpose(-1, -2) / math.sqrt(D), -1) @ v
    want = torch.softmax(k @ q.transpose(-1, -2) / math.sqrt(D), -1) @ z
    assert (Y.double() - want).norm() <= 5e-3 * want.norm()


def test_python_refusals():
    x = torch.zeros(2, 2, 8, 32, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(lengths=i32(1)), dict(lengths=torch.ones(2, device=DEV)), dict(documents=i32(1, 2)),
                dict(prefix=i32(1, 2)), dict(slopes=torch.ones(3, device=DEV)), dict(Y=x[:, :1].expand(2, 2, 8, 32)),
                dict(L_out=torch.ones(2, 2, 9, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            fl.flare_attention_fwd(x, x, x, **bad)
    for q, k, v in ((x.half(), x, x), (x, x[:, :, :4], x), (x[:, :, :, :24], x, x),
                    (torch.zeros(2, 3, 8, 32, dtype=torch.bfloat16, device=DEV), x, x), (x, x, x.cpu())):
        with pytest.raises((TypeError, ValueError)):
            fl.flare_attention_fwd(q, k, v)
    with pytest.raises(fl.FlareError):
        fl.flare_attention_fwd(x, x[:, :1].expand(2, 2, 8, 32), x)      # keys shared through a zero stride
    with pytest.raises(ValueError):
        fl.flare_attention_bwd(x, x, x, x, None, x)
