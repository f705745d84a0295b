"""Operators around the mixer where masks, epsilons, scales and memory are
unusual, against their definition in 64 bits."""
import math

import pytest
import torch

import rank_latent_routing_flare_b200 as fl

from . import attention_ref as ref
from .test_gpu_attention import DEV, check as check_poisoned, documents, i32, make, options
from .test_gpu_qk_norm_rope import STEP, angles, close, reference

pytestmark = pytest.mark.gpu


def hide_unseen(Q, K, V, dY, opts):
    """NaN and infinities in every key that no row sees and every row that sees no key."""
    B, _, Nq, _ = Q.shape
    masks = {n: opts[n] for n in ("lengths", "q_lengths", "q_offsets", "documents", "prefix", "causal") if n in opts}
    ok, _ = ref.visible(B, Nq, K.shape[2], DEV, **masks)
    no_key, no_row = ~ok.any(1).view(B, 1, -1, 1), ~ok.any(2).view(B, 1, -1, 1)
    for x, m, bad in ((K, no_key, math.nan), (V, no_key, math.inf), (Q, no_row, math.nan), (dY, no_row, -math.inf)):
        x.masked_fill_(m, bad)
    return Q, K, V, dY, opts


def check(Q, K, V, dY, opts, backward=True):
    want = ref.attention(Q, K, V, dY=dY if backward else None, **opts)
    Y, L = fl.flare_attention_fwd_train(Q, K, V, device_check=True, **opts)
    ref.close(Y, want["Y"], "Y")
    ref.close(L, want["L"], "L")
    if backward:
        for name, got in zip(("dQ", "dK", "dV"), fl.flare_attention_bwd(Q, K, V, Y, L, dY, device_check=True, **opts)):
            ref.close(got, want[name], name)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("N,cuts,dead,lengths", [
    (256, (60, 128), (1,), None),               # rows 60 .. 127 in no document: keys 64 .. 127 between two tiles' ranges
    (700, (60, 128, 316, 384), (1, 3), None),
    (2048, (1664, 1728), (), 100),              # documents beyond the length
    (2048, (40, 192, 1664, 1728), (1,), 1700),
])
def test_query_tiles_whose_keys_lie_apart(N, cuts, dead, lengths, D):
    """Keys between the ranges of a CTA's two query tiles, which neither of them takes part in."""
    o = {"documents": documents(2, N, cuts, dead)}
    if lengths:
        o["lengths"] = i32(lengths, N)
    for more in ({}, {"cap": 9.0}, {"bias": True}):
        check(*hide_unseen(*make(2, 2, 1, N, N, D, seed=N + D, **o, **more)), backward=not more)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
def test_few_rows_whose_document_lies_behind_the_length(D):
    """The last rows see nothing, their documents beginning behind lengths: what lies in between is padding."""
    ids = documents(2, 8, (5,))
    check_poisoned(*make(2, 1, 1, 8, 8, D, seed=41, documents=ids, lengths=i32(4, 2)), backward=False)
    ids = documents(2, 900, (300, 450, 700))
    for off in (i32(446, 296), i32(898, 697)):
        o = dict(documents=ids, lengths=i32(430, 777), q_offsets=off)
        check_poisoned(*make(2, 4, 2, 8, 900, D, seed=42, **o), backward=False)


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("slope", [0.3, 0.34, 0.35, 0.36])
@pytest.mark.parametrize("cap", [0.0, 120.0])
def test_a_large_score_at_the_far_end_of_a_tile(slope, cap, D):
    """Keys on either side of a tile's border outweigh all others, though the nearer of them is the farthest of its
    tile: the tile's largest product and its smallest distance belong to different keys."""
    N = 512
    Q, K, V, dY, _ = make(1, 2, 1, N, N, D, seed=D)
    Q.zero_()
    Q[..., 0] = 1
    o = {"slopes": torch.full((2,), slope, device=DEV), "causal": True, "scale": 1.0, "cap": cap}
    for border in (128, 256):
        for rivals, score in ((1, 48.5), (10, 49.0), (100, 49.0)):
            K.zero_()
            K[:, :, border, 0], K[:, :, border - rivals:border, 0] = 50.0, score
            check(Q, K, V, dY, o)


@pytest.mark.parametrize("slope", [0.02, 0.1, 0.3, 0.5])
def test_moderate_slopes_and_large_scores(slope):
    for D in (32, 128):
        Q, K, V, dY, _ = make(1, 4, 2, 700, 700, D, seed=40, qscale=12.0)
        check(Q, K, V, dY, {"slopes": slope * torch.tensor([1.0, 0.9, 1.1, -0.5], device=DEV), "causal": True})


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gain_gradients_without_an_epsilon(interleaved, D):
    """eps = 0: padding, and lanes without a row, add nothing to the gains' gradients."""
    g = torch.Generator(device=DEV).manual_seed(44)
    for B, N, H, lengths, shape in ((1, 1, 1, None, (D,)), (3, 37, 3, (37, 0, 5), (3, D)), (2, 700, 4, (699, 130), (D,))):
        x, dy = (torch.randn(B, H, N, D, generator=g, device=DEV).bfloat16() for _ in range(2))
        gain, freqs = 1 + 0.2 * torch.randn(shape, generator=g, device=DEV), torch.rand(D // 2, generator=g, device=DEV)
        n = None if lengths is None else i32(*lengths)
        got = fl.flare_qk_norm_rope_bwd(x, None, dy, None, gain, freqs=freqs, lengths=n, eps=0.0, interleaved=interleaved)
        want, tol = 0, 0
        for b in range(B):     # each entry's live rows on their own: the definition has no padding there
            m = N if lengths is None else lengths[b]
            if m:
                a = angles(m, freqs, None, 1)
                dx, dtol, dg, gt = reference(x[b:b + 1, :, :m], gain, a, None, 0.0, interleaved, dy=dy[b:b + 1, :, :m])
                close(got["dQ"][b:b + 1, :, :m], dx, dtol, "dQ")
                want, tol = want + dg, tol + gt
            assert (got["dQ"][b, :, m:] == 0).all()
        close(got["dq_gain"], want, tol * (1 + B * H * N * STEP) + B * H * N * STEP * want.abs(), "dq_gain")


UNSEEN = {
    # B, Hq, Hk, Nq, Nk, options
    "cache": (2, 4, 2, 1, 700, {"causal": True, "q_offsets": (300, 17)}),
    "cache_rows": (3, 4, 2, 4, 700, {"causal": True, "q_offsets": (300, 14, -2)}),
    "cache_documents": (2, 4, 2, 3, 700, {"documents": ((101, 333, 500), ()), "q_offsets": (120, 400)}),
    "cache_prefix": (2, 2, 2, 2, 700, {"causal": True, "prefix": (45, 333), "q_offsets": (20, 20)}),
    "chunk": (2, 4, 2, 200, 1500, {"causal": True, "q_offsets": (77, 900)}),
    "chunk_bias": (2, 4, 2, 200, 1500, {"causal": True, "q_offsets": (77, 900), "bias": True}),
    "chunk_cap": (2, 4, 2, 300, 700, {"causal": True, "q_offsets": (33, 100), "cap": 20.0, "prefix": (0, 450)}),
    "chunk_documents": (2, 4, 2, 300, 1500, {"documents": ((101, 333, 701), ()), "q_offsets": (120, 650)}),
    "chunk_padded": (2, 2, 1, 300, 600, {"causal": True, "q_offsets": (10, 200), "q_lengths": (140, 0),
                                         "lengths": (600, 300)}),
    "split": (1, 1, 1, 40, 5000, {"causal": True, "q_offsets": (3003,)}),
}


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("name", UNSEEN)
def test_keys_that_no_row_sees_may_hold_anything(name, D):
    """A cache's slots behind the newest token, other documents than the rows': as padding, they are not read into any
    result."""
    B, Hq, Hk, Nq, Nk, o = UNSEEN[name]
    check(*hide_unseen(*make(B, Hq, Hk, Nq, Nk, D, seed=Nk + D, **options(o, B, Nk))))


@pytest.mark.parametrize("D", [16, 128])
@pytest.mark.parametrize("Nk", [200, 1300])
@pytest.mark.parametrize("slope,off", [(4.0, 1 << 30), (-4.0, 1 << 30), (0.5, -(1 << 30)), (1e4, (1 << 31) - 200)])
def test_gradients_of_rows_far_from_their_keys(slope, off, Nk, D):
    """The distance that all keys of a row share is no part of its weights, however little of them it leaves in an
    fp32 log-sum-exp: every row's gradients are those of one that stands at its nearest key, as one more head does."""
    Nq = 40
    Q, K, V, dY, _ = make(2, 1, 1, Nq, Nk, D, seed=43, layout="head")
    if abs(slope) > 100:
        K.mul_(0.0)     # weights that the slope alone does not decide would need scores of its size
    o = {"slopes": torch.full((1,), slope, device=DEV), "q_offsets": i32(off, off), "lengths": i32(Nk, Nk // 3)}
    Y, L = fl.flare_attention_fwd_train(Q, K, V, **o)
    got = fl.flare_attention_bwd(Q, K, V, Y, L, dY, **o)
    near = i32(Nk - 1, Nk // 3 - 1) if off > 0 else i32(0, 0)
    folded = dict(slopes=torch.full((Nq,), slope, device=DEV), q_offsets=near, lengths=o["lengths"])
    rows = lambda t: t.transpose(1, 2)                                  # noqa: E731  (rows of one head as heads of one row)
    want = ref.attention(rows(Q), K, V, dY=rows(dY), **folded)
    ref.close(rows(Y), want["Y"], "Y")
    for name, g in zip(("dQ", "dK", "dV"), (rows(got[0]), *got[1:])):
        ref.close(g, want[name], name)


@pytest.mark.parametrize("D", [16, 128])
@pytest.mark.parametrize("scale,cap", [(1.0, 1e-6), (1e3, 1e-6), (1e4, 1e-2), (0.1, 1e-6), (30.0, 1e-4)])
def test_caps_far_below_the_scale(scale, cap, D):
    """Products bent from their last bits on: powers of scale / cap pass what fp32 holds."""
    for Nq in (2, 150):
        Q, K, V, dY, o = make(1, 2, 1, Nq, 200, D, seed=45, scale=scale, cap=cap)
        K[:, :, ::3] = 0.0                        # scores of exactly zero
        K[:, :, 1::3] *= 2.0 ** -20               # and some that the cap hardly bends
        check(Q, K, V, dY, o)
        K.mul_(0.0)                               # whole tiles of them
        check(Q, K, V, dY, o)


def test_gradients_that_arrive_off_a_16_byte_boundary():
    """Autograd hands over dense views of larger gradients, at any offset."""
    x = torch.randn(2, 2, 70, 32, device=DEV).bfloat16()
    gain, odd = torch.ones(32, device=DEV), torch.zeros(3, dtype=torch.bfloat16, device=DEV)
    w = torch.randn(3 + x.numel(), device=DEV).bfloat16()

    def grads(f, cut):
        leaf = x.clone().requires_grad_()
        y = f(leaf).reshape(-1)
        if cut:
            torch.cat((odd, y)).backward(w)        # y's gradient is w[3:]
        else:
            y.backward(w[3:].clone())
        return leaf.grad

    for f in (lambda t: fl.flare_attention(t, t, t, causal=True), lambda t: fl.flare_qk_norm_rope(t, None, gain)[0],
              lambda t: fl.flare_qk_norm_rope(None, t)[1]):
        assert torch.equal(grads(f, True), grads(f, False))


def test_learned_biases_and_angles_without_gradients():
    """Slopes, frequencies and positions that ask for gradients are refused only where gradients are recorded."""
    x = torch.randn(1, 2, 50, 32, device=DEV).bfloat16()
    slopes = torch.tensor([0.1, 0.2], device=DEV, requires_grad=True)
    freqs = torch.rand(2, 16, device=DEV, requires_grad=True)
    coords = torch.rand(1, 50, 2, device=DEV, requires_grad=True)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert torch.equal(fl.flare_attention(x, x, x, slopes=slopes), fl.flare_attention_fwd(x, x, x, slopes=slopes))
            assert torch.equal(fl.flare_qk_norm_rope(x, None, None, None, freqs, coords)[0],
                               fl.flare_qk_norm_rope_fwd(x, None, None, None, freqs, coords)[0])
    with pytest.raises(ValueError):
        fl.flare_attention(x, x, x, slopes=slopes)
    for f, p in ((freqs, coords.detach()), (freqs.detach(), coords)):
        with pytest.raises(ValueError):
            fl.flare_qk_norm_rope(x, None, None, None, f, p)


def test_memory_of_a_call_on_another_stream_is_not_taken_early():
    """A call on another stream does not write into memory that work queued on the current one still reads."""
    B, N, H, D = 1, 5000, 2, 64
    x = torch.randn(B, H, N, D, device=DEV).bfloat16()
    few, gain, freqs = x[:, :, :1], torch.ones(D, device=DEV), torch.rand(D // 2, device=DEV)
    Y, L = fl.flare_attention_fwd_train(x, x, x)
    side = torch.cuda.Stream()
    calls = {
        "rows": lambda: fl.flare_qk_norm_rope_fwd(x, x, gain, gain, freqs, stream=side),
        "gradients": lambda: fl.flare_qk_norm_rope_bwd(x, x, x, x, gain, gain, freqs, stream=side),
        "attention": lambda: fl.flare_attention_fwd_train(x, x, x, stream=side),
        "few": lambda: fl.flare_attention_fwd(few, x, x, stream=side),
        "backward": lambda: fl.flare_attention_bwd(x, x, x, Y, L, x, stream=side),
    }
    sizes = [x.numel() * 2, L.numel() * 4, gain.numel() * 4, few.numel() * 2, 256,
             fl.flare_attention_workspace_bytes(B, H, H, N, N, D), fl.flare_attention_workspace_bytes(B, H, H, 1, N, D),
             fl.flare_attention_workspace_bytes(B, H, H, N, N, D, True), fl.flare_qk_norm_rope_workspace_bytes(B, N, H, H, D)]
    for name, call in calls.items():
        call()
        torch.cuda.synchronize()
        held = [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
        copies = [torch.empty_like(t) for t in held]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)                                   # some 20 ms
        for c, t in zip(copies, held):
            c.copy_(t)
        del held, c, t                                                  # freed, and still to be read
        out = call()
        torch.cuda.synchronize()
        assert all((c == 77).all() for c in copies), name
        del out


def test_gains_off_a_16_byte_boundary_are_named():
    x = torch.randn(1, 2, 40, 32, device=DEV).bfloat16()
    off, ok = torch.ones(33, device=DEV)[1:], torch.ones(32, device=DEV)
    for bad in (dict(Q=x, q_gain=off), dict(K=x, k_gain=off), dict(K=x, k_gain=torch.ones(65, device=DEV)[1:].view(2, 32))):
        with pytest.raises(ValueError, match="_gain.*16-byte"):
            fl.flare_qk_norm_rope_fwd(**bad)
    with pytest.raises(ValueError, match="dq_gain.*16-byte"):
        fl.flare_qk_norm_rope_bwd(x, None, x, None, ok, grads={"dq_gain": torch.empty(33, device=DEV)[1:]})


def test_mixer_and_split_attention_at_once():
    """The mixer's kernels and attention whose clusters join their splits, on two streams: neither waits for columns
    of TMEM that the other holds until a third has run."""
    g = torch.Generator(device=DEV).manual_seed(46)
    K, V = (torch.randn(1, 8, 60000, 16, generator=g, device=DEV).bfloat16() for _ in range(2))
    latents = torch.randn(8, 64, 16, generator=g, device=DEV).bfloat16()
    jobs = [make(1, 4, 2, 512, 2000, 32, seed=47), make(1, 8, 1, 700, 700, 32, seed=48, causal=True),
            make(1, 8, 1, 700, 700, 64, seed=49, causal=True), make(1, 2, 2, 600, 1500, 64, seed=50)]

    def attend():
        out = []
        for Q, k, v, dY, o in jobs:
            Y, L = fl.flare_attention_fwd_train(Q, k, v, **o)
            out += [Y, L, *fl.flare_attention_bwd(Q, k, v, Y, L, dY, **o)]
        return out

    want, mixed = attend(), fl.flare_mixer_fwd(K, V, latents, device_check=False)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s in streams[:2]:
            with torch.cuda.stream(s):
                got.append(attend())
        with torch.cuda.stream(streams[2]):
            ys = [fl.flare_mixer_fwd(K, V, latents, device_check=False) for _ in range(6)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x in got for a, b in zip(x, want)) and all(torch.equal(y, mixed) for y in ys)
