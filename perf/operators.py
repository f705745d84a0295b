"""Cases of the operators around the mixer: the preparation of queries and
keys (per-head norm and position rotation) and exact softmax attention with
capped scores, a distance bias and packed-document, prefix and padding masks.

``run`` computes a case in its plain form (elementary torch operations in
fp32, angles in fp64) or, with ``own`` set, through the package's entry points.
"""
import math

import torch

own = False


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def _prep(name, op, B, N, Hq, Hk, D, pos, gain, interleaved=False, ragged=False, rot=None):
    return {"name": name, "op": op, "B": B, "N": N, "Hq": Hq, "Hk": Hk, "D": D, "pos": pos, "gain": gain,
            "interleaved": interleaved, "ragged": ragged, "rot": D if rot is None else rot}


def _attn(name, op, B, Hq, Hk, Nq, Nk, D, causal=False, docs=0, prefix=False, ragged=False, bias=False, cap=0.0):
    return {"name": name, "op": op, "B": B, "Hq": Hq, "Hk": Hk, "Nq": Nq, "Nk": Nk, "D": D, "causal": causal,
            "docs": docs, "prefix": prefix, "ragged": ragged, "bias": bias, "cap": cap}


def listed():
    return [
        # the queries and keys of one new token of 32 sequences, grouped heads: a serving step, all latency
        _prep("prep_step_b32", "prep_fwd", 32, 1, 32, 8, 128, "int", "shared"),
        # the keys of a million-point mesh, rotated by its 3-D coordinates, before the fixed-query mixer reads them
        _prep("prep_keys_mesh_1m", "prep_fwd", 1, 1 << 20, 0, 8, 16, "coord3", "head"),
        # a padded batch of 4K-token sequences, queries and keys, partly rotated
        _prep("prep_fwd_padded_4k", "prep_fwd", 32, 4096, 8, 8, 32, "int", "shared", ragged=True, rot=16),
        # the same preparation's gradients in training, grouped heads, an odd length
        _prep("prep_bwd_gqa_8191", "prep_bwd", 2, 8191, 32, 8, 128, "int", "shared", interleaved=True),
        # gradients of the small heads over points with 2-D coordinates
        _prep("prep_bwd_points_65k", "prep_bwd", 4, 65536, 8, 8, 16, "coord2", "head"),
        # a small unmasked mixer-sized call: latency and exponentials
        _attn("attn_small_1k", "attn_fwd", 1, 4, 4, 1024, 1024, 16),
        # packed documents with capped scores, grouped heads
        _attn("attn_docs_cap_8k", "attn_fwd", 2, 16, 4, 8192, 8192, 64, causal=True, docs=12, cap=30.0),
        # one long causal sequence with a distance bias
        _attn("attn_causal_bias_16k", "attn_fwd", 1, 8, 2, 16384, 16384, 128, causal=True, bias=True),
        # training on a padded batch of the masked workload's shape, no other mask
        _attn("attn_train_padded_4k", "attn_train", 8, 8, 8, 4096, 4096, 32, ragged=True),
        # training with a bidirectional prefix at an odd length, grouped heads, capped scores
        _attn("attn_train_prefix_cap_4095", "attn_train", 2, 16, 4, 4095, 4095, 128, causal=True, prefix=True,
              cap=50.0),
        # one new token of 16 sequences over long caches of ragged lengths
        _attn("attn_step_32k", "attn_fwd", 16, 32, 8, 1, 32768, 128, causal=True, ragged=True),
        # one new token over a short cache: latency
        _attn("attn_step_513", "attn_fwd", 1, 8, 8, 1, 513, 32, causal=True, ragged=True, bias=True, cap=30.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep_fwd", "prep_bwd", "attn_fwd", "attn_train", "attn_step"])
    D = rng.choice([16, 32, 64, 128])
    Hk = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 1, 2, 4])
    if op.startswith("prep"):
        heads = Hk * (group + 1)
        most = (1 << 26) // (heads * D)
        B = rng.choice([1, 2, 5, 8, 32])
        N = _log_int(rng, 1, max(2, min(1 << 20, most // B)))
        rot = rng.choice([D, D, D // 2]) if D >= 32 else D
        return _prep("", op, B, N, Hk * group, Hk, D, rng.choice(["none", "int", "coord2", "coord3"]),
                     rng.choice(["none", "shared", "head"]), rng.random() < 0.5, rng.random() < 0.4, rot)
    B = rng.choice([1, 2, 3, 8])
    causal = rng.random() < 0.6
    extra = {"ragged": rng.random() < 0.4, "bias": rng.random() < 0.4, "cap": rng.choice([0.0, 0.0, 20.0, 50.0])}
    if op == "attn_step":
        Nk = _log_int(rng, 1, min(65536, (1 << 28) // (B * Hk * D)))
        Nq = rng.choice([1, 1, 1, 2, 4])
        return _attn("", "attn_fwd", B, Hk * group, Hk, Nq, max(Nk, Nq), D, causal=True, **extra)
    pairs = (1 << 30) // (B * Hk * group) if op == "attn_fwd" else (1 << 29) // (B * Hk * group)
    N = _log_int(rng, 1, min(16384, math.isqrt(pairs)))
    Nq = N if causal or rng.random() < 0.5 else _log_int(rng, 1, N)
    docs = rng.choice([0, 0, 3, 9]) if Nq == N and N >= 16 else 0
    return _attn("", op, B, Hk * group, Hk, Nq, N, D, causal=causal, docs=docs,
                 prefix=causal and not docs and rng.random() < 0.5, **extra)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _heads(packed, B, N, first, H, D):
    """Heads [first, first + H) of a packed token-major projection, as a [B, H, N, D] view."""
    return packed.view(B, N, -1, D)[:, :, first:first + H].transpose(1, 2)


def _prepare_prep(c, g):
    dev = "cuda"
    B, N, Hq, Hk, D = c["B"], c["N"], c["Hq"], c["Hk"], c["D"]
    # queries, keys and values as one projection of the tokens writes them: the operator reads slices of it
    Ht = Hq + 2 * Hk
    packed = torch.empty(B, N, Ht * D, dtype=torch.bfloat16, device=dev).normal_(0.0, 1.3, generator=g)
    s = {"c": c, "Q": _heads(packed, B, N, 0, Hq, D) if Hq else None, "K": _heads(packed, B, N, Hq, Hk, D)}
    shape = {"none": None, "shared": lambda H: (D,), "head": lambda H: (H, D)}[c["gain"]]
    for key, H in (("q_gain", Hq), ("k_gain", Hk)):
        s[key] = None if shape is None or not H else 1.0 + 0.2 * torch.randn(shape(H), generator=g, device=dev)
    P = c["rot"] // 2
    axis = {"none": 1, "int": 1, "coord2": 2, "coord3": 3}[c["pos"]]
    if c["pos"] in ("none", "int"):
        # a geometric ladder of frequencies over integer positions
        s["freqs"] = (500000.0 ** (-torch.arange(P, device=dev, dtype=torch.float64) / P)).float().view(1, P)
        s["positions"] = None
        if c["pos"] == "int":
            start = torch.randint(0, 1 << 17, (B, 1), generator=g, device=dev, dtype=torch.int32)
            s["positions"] = start + torch.arange(N, device=dev, dtype=torch.int32)
    else:
        # points of the unit square or cube; every pair mixes the axes with its own wave numbers
        s["freqs"] = torch.randn(axis, P, generator=g, device=dev) * 2.0 ** (torch.arange(P, device=dev) % 7)
        s["positions"] = torch.rand(B, N, axis, generator=g, device=dev)
    s["lengths"] = torch.randint(max(1, N // 4), N + 1, (B,), generator=g, device=dev, dtype=torch.int32) \
        if c["ragged"] else None
    if c["op"] == "prep_bwd":
        for key, H in (("dQr", Hq), ("dKr", Hk)):
            s[key] = torch.empty(B, H, N, D, dtype=torch.bfloat16, device=dev).normal_(generator=g) if H else None
    return s


def _prepare_attn(c, g):
    dev = "cuda"
    B, Hq, Hk, Nq, Nk, D = c["B"], c["Hq"], c["Hk"], c["Nq"], c["Nk"], c["D"]
    bf = dict(dtype=torch.bfloat16, device=dev)
    s = {"c": c, "lengths": None, "q_lengths": None, "q_offsets": None, "documents": None, "prefix": None,
         "slopes": None}
    if Nq == Nk:
        # queries and keys head-major, as the preparation writes them; values a slice of the packed projection
        s["Q"] = torch.empty(B, Hq, Nq, D, **bf).normal_(0.0, 1.5, generator=g)
        s["K"] = torch.empty(B, Hk, Nk, D, **bf).normal_(generator=g)
        packed = torch.empty(B, Nk, 2 * Hk * D, **bf).normal_(generator=g)
        s["V"] = _heads(packed, B, Nk, Hk, Hk, D)
    else:
        # new tokens (or other queries) against keys and values kept head-major
        s["Q"] = _heads(torch.empty(B, Nq, Hq * D, **bf).normal_(0.0, 1.5, generator=g), B, Nq, 0, Hq, D)
        s["K"] = torch.empty(B, Hk, Nk, D, **bf).normal_(generator=g)
        s["V"] = torch.empty(B, Hk, Nk, D, **bf).normal_(generator=g)
    if c["ragged"]:
        n = torch.randint(max(Nq if Nq < Nk else 1, Nk // 4), Nk + 1, (B,), generator=g, device=dev,
                          dtype=torch.int32)
        s["lengths"] = n
        if Nq == Nk:
            s["q_lengths"] = n
        elif c["causal"]:
            s["q_offsets"] = n - Nq          # the new tokens are the last of each cache
    if c["docs"]:
        cuts = torch.randint(0, Nk, (B, c["docs"] - 1), generator=g, device=dev)
        s["documents"] = torch.zeros(B, Nk, dtype=torch.int32, device=dev).scatter_add_(
            1, cuts, torch.ones_like(cuts, dtype=torch.int32)).cumsum(1, dtype=torch.int32)
    if c["prefix"]:
        s["prefix"] = torch.randint(0, Nk // 2 + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    if c["bias"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq)
    if c["op"] == "attn_train":
        s["dY"] = torch.empty(B, Hq, Nq, D, **bf).normal_(generator=g)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return _prepare_prep(case, g) if case["op"].startswith("prep") else _prepare_attn(case, g)


# ----------------------------------------------------------------------------
# preparation of queries and keys: plain form
# ----------------------------------------------------------------------------

def _angles(s):
    """cos and sin of position x frequency, [B or 1, 1, N, P] in fp32, the angle itself in fp64."""
    c = s["c"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(c["N"], device="cuda").view(1, -1, 1)
    elif pos.dim() == 2:
        pos = pos.unsqueeze(-1)
    a = torch.matmul(pos.double(), s["freqs"].double()).unsqueeze(1)
    return a.cos().float(), a.sin().float()


def _pairs(x, c):
    """The two members of every rotated pair, and the elements that are not rotated."""
    R = c["rot"]
    if c["interleaved"]:
        return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]
    return x[..., :R // 2], x[..., R // 2:R], x[..., R:]


def _join(a, b, rest, c):
    ab = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((ab, rest), -1) if rest.shape[-1] else ab


def _live_rows(lengths, N):
    return None if lengths is None else (torch.arange(N, device="cuda") < lengths.view(-1, 1)).view(-1, 1, N, 1)


def _gain(g):
    return None if g is None else g if g.dim() == 1 else g.unsqueeze(1)


EPS = 1e-6


def _prep_fwd_plain(x, gain, cos, sin, live, c):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    if gain is not None:
        y = y * _gain(gain)
    a, b, rest = _pairs(y, c)
    y = _join(a * cos - b * sin, a * sin + b * cos, rest, c)
    if live is not None:
        y = y * live
    return y.to(torch.bfloat16)


def _prep_bwd_plain(x, gain, dy, cos, sin, live, c):
    x, dy = x.float(), dy.float()
    if live is not None:
        dy = dy * live
    a, b, rest = _pairs(dy, c)
    u = _join(a * cos + b * sin, b * cos - a * sin, rest, c)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    dgain = None
    if gain is not None:
        dgain = (u * n).sum((0, 2) if gain.dim() == 2 else (0, 1, 2))
        u = u * _gain(gain)
    dx = r * (u - n * (u * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dgain


def _run_prep(s):
    c = s["c"]
    if own:
        import rank_latent_routing_flare_b200 as fl
        opts = dict(freqs=s["freqs"], positions=s["positions"], lengths=s["lengths"], eps=EPS,
                    interleaved=c["interleaved"])
        if c["op"] == "prep_fwd":
            Qr, Kr = fl.flare_qk_norm_rope_fwd(s["Q"], s["K"], s["q_gain"], s["k_gain"], **opts)
            return {"Q": Qr, "K": Kr}
        return fl.flare_qk_norm_rope_bwd(s["Q"], s["K"], s["dQr"], s["dKr"], s["q_gain"], s["k_gain"],
                                         **opts)
    cos, sin = _angles(s)
    live = _live_rows(s["lengths"], c["N"])
    out = {}
    for x, gain in (("Q", "q_gain"), ("K", "k_gain")):
        if s[x] is None:
            continue
        if c["op"] == "prep_fwd":
            out[x] = _prep_fwd_plain(s[x], s[gain], cos, sin, live, c)
        else:
            out["d" + x], out["d" + gain] = _prep_bwd_plain(s[x], s[gain], s["d" + x + "r"], cos, sin, live, c)
    return out


# ----------------------------------------------------------------------------
# attention: plain form
# ----------------------------------------------------------------------------

def _positions_of_queries(s):
    c = s["c"]
    off = s["q_offsets"]
    off = torch.full((c["B"],), c["Nk"] - c["Nq"], device="cuda") if off is None else off
    return off.view(-1, 1) + torch.arange(c["Nq"], device="cuda")                      # [B, Nq]


def _runs(ids):
    """Index of the run of equal ids that each position lies in; -1 where the id is negative."""
    new = torch.zeros_like(ids)
    new[:, 1:] = ids[:, 1:] != ids[:, :-1]
    return new.cumsum(1).masked_fill(ids < 0, -1)


def _banned(s):
    """True where a query may not see a key, [B, Nq, Nk]; None without any mask."""
    c = s["c"]
    p = _positions_of_queries(s).unsqueeze(-1)
    j = torch.arange(c["Nk"], device="cuda")
    ban = None
    if c["causal"]:
        ban = j > p
        if s["prefix"] is not None:
            ban &= j >= s["prefix"].view(-1, 1, 1)
    for n, at in ((s["lengths"], j), (s["q_lengths"], torch.arange(c["Nq"], device="cuda").unsqueeze(-1))):
        if n is not None:
            out = at >= n.view(-1, 1, 1)
            ban = out if ban is None else ban | out
    if s["documents"] is not None:
        run = _runs(s["documents"])
        mine = run.gather(1, p.squeeze(-1).clamp(0, c["Nk"] - 1).long()).unsqueeze(-1)
        out = (mine != run.unsqueeze(1)) | (mine < 0) | (p < 0) | (p >= c["Nk"])
        ban = out if ban is None else ban | out
    return ban


def _scores(s, q, k):
    """Scores before the mask, [B, Hk, G, Nq, Nk], and tanh of the capped ones (None without a cap)."""
    c = s["c"]
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(c["D"]))
    t = None
    if c["cap"]:
        t = x.mul_(1.0 / c["cap"]).tanh_()
        x = t * c["cap"]
    if s["slopes"] is not None:
        p = _positions_of_queries(s).unsqueeze(-1)
        dist = (p - torch.arange(c["Nk"], device="cuda")).abs().float()
        x = x - s["slopes"].view(1, c["Hk"], -1, 1, 1) * dist.view(-1, 1, 1, c["Nq"], c["Nk"])
    return x, t


def _run_attn(s):
    c = s["c"]
    B, Hq, Hk, Nq, Nk, D = c["B"], c["Hq"], c["Hk"], c["Nq"], c["Nk"], c["D"]
    train = c["op"] == "attn_train"
    if own:
        import rank_latent_routing_flare_b200 as fl
        opts = dict(lengths=s["lengths"], q_lengths=s["q_lengths"], q_offsets=s["q_offsets"],
                    documents=s["documents"], prefix=s["prefix"], slopes=s["slopes"], causal=c["causal"],
                    cap=c["cap"])
        if not train:
            return fl.flare_attention_fwd(s["Q"], s["K"], s["V"], **opts)
        Y, L = fl.flare_attention_fwd_train(s["Q"], s["K"], s["V"], **opts)
        dQ, dK, dV = fl.flare_attention_bwd(s["Q"], s["K"], s["V"], Y, L, s["dY"], **opts)
        return {"Y": Y, "L": L, "dQ": dQ, "dK": dK, "dV": dV}
    q = s["Q"].float().reshape(B, Hk, Hq // Hk, Nq, D)
    k, v = s["K"].float().unsqueeze(2), s["V"].float().unsqueeze(2)
    x, t = _scores(s, q, k)
    ban = _banned(s)
    if ban is not None:
        ban = ban.view(-1, 1, 1, Nq, Nk)
        x.masked_fill_(ban, -math.inf)
    top = x.amax(-1, keepdim=True)
    base = top.masked_fill(top == -math.inf, 0.0)
    e = x.sub_(base).exp_()
    total = e.sum(-1, keepdim=True)
    p = e.div_(total.masked_fill(total == 0, 1.0))
    y = torch.matmul(p, v)
    Y = y.reshape(B, Hq, Nq, D).to(torch.bfloat16)
    if not train:
        return Y
    L = (base + total.log()).reshape(B, Hq, Nq)
    dy = s["dY"].float().reshape(B, Hk, Hq // Hk, Nq, D)
    dv = torch.matmul(p.transpose(-1, -2), dy).sum(2)
    ds = torch.matmul(dy, v.transpose(-1, -2)).sub_((dy * y).sum(-1, keepdim=True)).mul_(p)
    if t is not None:
        ds.mul_(t.square_().neg_().add_(1.0))
    ds.mul_(1.0 / math.sqrt(D))
    dq = torch.matmul(ds, k).reshape(B, Hq, Nq, D)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return {"Y": Y, "L": L, "dQ": dq.to(torch.bfloat16), "dK": dk.to(torch.bfloat16), "dV": dv.to(torch.bfloat16)}


def run(state):
    return _run_prep(state) if state["c"]["op"].startswith("prep") else _run_attn(state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"].startswith("prep"):
        valid = 0.625 if c["ragged"] else 1.0                  # lengths are uniform in [N / 4, N]
        tok, H = c["B"] * c["N"], c["Hq"] + c["Hk"]
        rows = 2 * tok * H * c["D"]                            # bf16 rows of the queries and keys
        pos = {"none": 0, "int": 4, "coord2": 8, "coord3": 12}[c["pos"]] * tok * valid
        reads = 1 if c["op"] == "prep_fwd" else 2              # x; x and the gradient; rows of padding are written only
        # per element: square, norm, gain, rotation (3 products and sums); the gradient twice that
        return {"bytes": rows * (reads * valid + 1) + pos, "flops": (8 if c["op"] == "prep_fwd" else 16) * tok * H *
                c["D"] * valid}
    B, Hq, Hk, Nq, Nk, D = c["B"], c["Hq"], c["Hk"], c["Nq"], c["Nk"], c["D"]
    live_k = 0.625 if c["ragged"] else 1.0
    live_q = live_k if Nq == Nk else 1.0
    pairs = (0.4375 if Nq == Nk and c["ragged"] else live_k) * Nq * Nk
    if c["docs"]:
        pairs *= 2.0 / (c["docs"] + 1)                         # expected sum of squares of random document lengths
    if c["causal"] and Nq == Nk:
        pairs *= 0.5 * (1 + 1 / 12 if c["prefix"] else 1)      # a prefix uniform in [0, N / 2] adds N^2 / 24
    qrows, krows = 2 * B * Hq * Nq * D, 2 * B * Hk * Nk * D
    bytes_ = qrows * live_q + 2 * krows * live_k + qrows       # Q, K, V in, Y out
    flops = 4 * D * B * Hq * pairs
    if c["op"] == "attn_train":                                # dY in, L, dQ, dK, dV out; five more products
        bytes_ += qrows * live_q + 4 * B * Hq * Nq + qrows + 2 * krows
        flops *= 3.5
    return {"bytes": bytes_, "flops": flops}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

def _exact_prep(s):
    c = s["c"]
    B, N, D, R = c["B"], c["N"], c["D"], c["rot"]
    P = R // 2
    first = torch.arange(P, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else P)
    pos = torch.arange(N, device="cuda").expand(B, N) if s["positions"] is None else s["positions"]
    pos = pos.double().reshape(B, N, -1)
    angle = sum(pos[:, :, a, None] * s["freqs"].double()[a] for a in range(pos.shape[-1]))      # [B, N, P]
    turn = torch.polar(torch.ones_like(angle), angle)
    out = {}
    for key, gk in (("Q", "q_gain"), ("K", "k_gain")):
        if s[key] is None:
            continue
        H = s[key].shape[1]
        res = torch.zeros(B, H, N, D, dtype=torch.float64, device="cuda")
        gain = None if s[gk] is None else s[gk].double().expand(H, D)
        dgain = torch.zeros(H, D, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = N if s["lengths"] is None else int(s["lengths"][b])
            for h in range(H):
                x = s[key][b, h, :n].double()
                norm = (x.pow(2).sum(1) / D + EPS).sqrt().unsqueeze(1)
                unit = x / norm
                w = torch.ones(D, dtype=torch.float64, device="cuda") if gain is None else gain[h]
                z = unit * w if c["op"] == "prep_fwd" else s["d" + key + "r"][b, h, :n].double()
                spin = turn[b, :n] if c["op"] == "prep_fwd" else turn[b, :n].conj()
                pair = torch.complex(z[:, first], z[:, second]) * spin
                z = z.clone()
                z[:, first], z[:, second] = pair.real, pair.imag
                if c["op"] == "prep_bwd":
                    dgain[h] += (z * unit).sum(0)
                    z = z * w
                    z = (z - unit * ((z * unit).sum(1, keepdim=True) / D)) / norm
                res[b, h, :n] = z
        if c["op"] == "prep_fwd":
            out[key] = res
        else:
            out["d" + key] = res
            out["d" + gk] = None if gain is None else dgain if s[gk].dim() == 2 else dgain.sum(0)
    return out


def _exact_attn(s):
    c = s["c"]
    B, Hq, Hk, Nq, Nk, D = c["B"], c["Hq"], c["Hk"], c["Nq"], c["Nk"], c["D"]
    f64 = dict(dtype=torch.float64, device="cuda")
    train = c["op"] == "attn_train"
    Y = torch.zeros(B, Hq, Nq, D, **f64)
    L, dQ = torch.full((B, Hq, Nq), -math.inf, **f64), torch.zeros_like(Y)
    dK, dV = torch.zeros(B, Hk, Nk, D, **f64), torch.zeros(B, Hk, Nk, D, **f64)
    i, j = torch.arange(Nq, device="cuda"), torch.arange(Nk, device="cuda")
    for b in range(B):
        at = i + (Nk - Nq if s["q_offsets"] is None else int(s["q_offsets"][b]))
        # every mask here leaves a query one interval [lo, hi) of keys
        lo, hi = torch.zeros_like(i), torch.full_like(i, Nk if s["lengths"] is None else int(s["lengths"][b]))
        if c["causal"]:
            see = at + 1
            if s["prefix"] is not None:
                see = see.clamp(min=int(s["prefix"][b]))
            hi = torch.minimum(hi, see)
        if s["documents"] is not None:
            ids = s["documents"][b].tolist()
            start, end = list(range(Nk)), list(range(1, Nk + 1))
            for n in range(1, Nk):
                if ids[n] == ids[n - 1]:
                    start[n] = start[n - 1]
            for n in range(Nk - 2, -1, -1):
                if ids[n] == ids[n + 1]:
                    end[n] = end[n + 1]
            there = at.clamp(0, Nk - 1)
            lo = torch.tensor(start, device="cuda")[there]
            hi = torch.minimum(hi, torch.tensor(end, device="cuda")[there])
        if s["q_lengths"] is not None:
            hi = torch.where(i < int(s["q_lengths"][b]), hi, lo)
        ok = (j >= lo.unsqueeze(1)) & (j < hi.unsqueeze(1))
        some = ok.any(1)
        for h in range(Hq):
            kv = h // (Hq // Hk)
            q, k, v = s["Q"][b, h].double(), s["K"][b, kv].double(), s["V"][b, kv].double()
            z = q @ k.T / math.sqrt(D)
            if c["cap"]:
                z = torch.tanh(z / c["cap"])
                slope = 1 - z * z
                z = c["cap"] * z
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double() * (at.unsqueeze(1) - j).abs()
            z = torch.where(ok, z, -math.inf)
            norm = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.where(some, norm, 0.0).unsqueeze(1))
            Y[b, h], L[b, h] = p @ v, norm
            if train:
                dy = s["dY"][b, h].double()
                dV[b, kv] += p.T @ dy
                dp = dy @ v.T
                dz = p * (dp - (p * dp).sum(1, keepdim=True))
                if c["cap"]:
                    dz = dz * slope
                dQ[b, h] = dz @ k / math.sqrt(D)
                dK[b, kv] += dz.T @ q / math.sqrt(D)
    return {"Y": Y, "L": L, "dQ": dQ, "dK": dK, "dV": dV} if train else Y


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_prep(s) if case["op"].startswith("prep") else _exact_attn(s)
