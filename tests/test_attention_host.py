"""Host-only checks of the attention's entry points: refusals come back before
anything is enqueued, workspaces are sized from the shapes alone; and the
64-bit reference of the GPU tests against autograd and differences."""
import os
import re

import pytest
import torch

import rank_latent_routing_flare_b200 as fl
from rank_latent_routing_flare_b200 import Status
from rank_latent_routing_flare_b200 import attention as m

from . import attention_ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "flare_ops.h")
A, W = 0x10000, 0x20000   # never dereferenced: every call fails a check, or finds no device

NAMES = (["B", "Hq", "Hk", "Nq", "Nk", "D", "causal", "scale", "cap"]
         + [n + s for n in ("Q", "K", "V") for s in ("", "0", "1", "2")]
         + ["lengths", "q_lengths", "q_offsets", "documents", "prefix", "slopes", "Y", "Y0", "Y1", "Y2", "L"]
         + [n + s for n in ("dY", "dQ", "dK", "dV") for s in ("", "0", "1", "2")])


def args(**over):
    v = dict.fromkeys(NAMES, 0)
    v.update(B=2, Hq=4, Hk=2, Nq=100, Nk=300, D=32, scale=0.0, cap=0.0, L=A)
    for x, H, N in (("Q", 4, 100), ("K", 2, 300), ("V", 2, 300), ("Y", 4, 100), ("dY", 4, 100), ("dQ", 4, 100),
                    ("dK", 2, 300), ("dV", 2, 300)):
        v[x], v[x + "0"], v[x + "1"], v[x + "2"] = A, H * N * 32, N * 32, 32
    v.update(over)
    return m._ARGS.pack(*[v[n] for n in NAMES])


def fwd(ws=W, ws_bytes=1 << 40, **over):
    return fl.load_library().flare_attention_fwd(args(**over), ws, ws_bytes, None)


def bwd(ws=W, ws_bytes=1 << 40, **over):
    return fl.load_library().flare_attention_bwd(args(**over), ws, ws_bytes, None)


def test_struct_matches_the_packing():
    text = open(HEADER).read()
    body = re.search(r"typedef struct \{((?:(?!typedef).)*?)\} flare_attention_args;", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    members = sum(3 if "[3]" in d else 1 for line in body.split(";") for d in line.split(",") if d.strip())
    assert members == len(NAMES) and m._ARGS.size == 8 * members


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(call):
    for over in (dict(Q=0), dict(V=0), dict(Y=0), dict(ws=None)):
        assert call(**over) == Status.ERR_NULL, over
    for over in (dict(Nq=0), dict(B=0), dict(Hq=3), dict(Hk=0), dict(prefix=A), dict(cap=float("nan")),
                 dict(scale=float("inf")), dict(K2=8), dict(Q1=-3200)):
        assert call(**over) == Status.ERR_SHAPE, over
    for over in (dict(D=48), dict(D=256), dict(Nk=1 << 31), dict(B=70000), dict(K0=0), dict(Q2=0)):
        assert call(**over) == Status.ERR_UNSUPPORTED, over
    for over in (dict(Q=A + 8), dict(V2=36), dict(lengths=A + 2), dict(L=A + 1), dict(ws=W + 16), dict(Y=A + 4)):
        assert call(**over) == Status.ERR_ALIGN, over
    need = fl.flare_attention_workspace_bytes(2, 4, 2, 100, 300, 32, backward=call is bwd)
    assert call(ws_bytes=need - 1) == Status.ERR_WORKSPACE


@pytest.mark.parametrize("call", [fwd, bwd])
def test_caps_and_lengths_out_of_range(call):
    for over in (dict(cap=1e-7), dict(cap=1e10), dict(cap=1e-60), dict(Nk=(1 << 27) + 1), dict(Nq=(1 << 27) + 1)):
        assert call(**over) == Status.ERR_UNSUPPORTED, over
    for over in (dict(cap=1e-6), dict(cap=1e9), dict(cap=-1e30)):
        assert call(**over) != Status.ERR_UNSUPPORTED, over


def test_backward_refusals():
    for name in ("L", "dY", "dQ", "dK", "dV"):
        assert bwd(**{name: 0}) == Status.ERR_NULL, name
    assert bwd(dK1=0) == Status.ERR_SHAPE and bwd(dY0=0) == Status.ERR_UNSUPPORTED
    lib = fl.load_library()
    assert lib.flare_attention_fwd(None, W, 1 << 40, None) == Status.ERR_NULL
    assert lib.flare_attention_bwd(None, W, 1 << 40, None) == Status.ERR_NULL


def test_workspace_sizes():
    f = fl.flare_attention_workspace_bytes
    assert f(1, 8, 8, 1, 32768, 128) >= 2 * 8 * 129 * 4             # one token over a long cache: split and joined
    assert f(2, 4, 2, 100, 300, 32, backward=True) > 2 * 4 * 100 * 16
    assert f(4, 32, 8, 8192, 8192, 128) % 256 == 0
    for bad in ((0, 1, 1, 1, 1, 16), (1, 3, 2, 1, 1, 16), (1, 1, 1, 1, 1, 24), (1, 1, 1, 0, 1, 16)):
        assert f(*bad) == 0


def test_valid_calls_reach_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the pointers are not real")
    assert fwd() == Status.ERR_LAUNCH and bwd() == Status.ERR_LAUNCH
    assert fwd(L=0) == Status.ERR_LAUNCH                             # the sums are optional in the forward
    assert fwd(B=1, Hq=1, Hk=1, Nq=1, Nk=1, Q0=0, K0=0, Q1=3, K2=0) == Status.ERR_LAUNCH   # strides of size one are not read


def test_python_refusals():
    x = torch.zeros(1, 2, 3, 16, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fl.flare_attention_fwd(x, x, x)
    with pytest.raises(ValueError):
        fl.flare_attention_fwd(x[0], x, x)


@pytest.mark.parametrize("cap,bias,causal", [(0.0, False, False), (3.0, True, True)])
def test_reference_gradients(cap, bias, causal):
    """The reference's gradients against autograd through its own forward, and against differences."""
    g = torch.Generator().manual_seed(0)
    B, Hq, Hk, N, D = 2, 4, 2, 13, 16
    q, k, v, dy = (torch.randn(B, H, N, D, generator=g, dtype=torch.float64) for H in (Hq, Hk, Hk, Hq))
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0]) if bias else None
    opts = dict(cap=cap, slopes=slopes, causal=causal, lengths=torch.tensor([13, 6]), q_lengths=torch.tensor([13, 6]),
                documents=torch.tensor([[0] * 5 + [1] * 8, [4] * 6 + [-1] * 7]))
    ref = attention_ref.attention(q, k, v, dY=dy, **opts)
    f = lambda a, b, c: (attention_ref.attention(a, b, c, **opts)["Y"][0] * dy).sum()   # noqa: E731
    for n, key in enumerate(("dQ", "dK", "dV")):
        ts = [q, k, v]
        step = torch.randn(ts[n].shape, generator=g, dtype=torch.float64)
        up, down = list(ts), list(ts)
        up[n], down[n] = ts[n] + 1e-5 * step, ts[n] - 1e-5 * step
        want = (f(*up) - f(*down)) / 2e-5
        assert abs((ref[key][0] * step).sum() - want) <= 1e-7 * (1 + abs(want))
    assert (ref["Y"][0][1, :, 6:] == 0).all() and (ref["L"][0][1, :, 6:] == float("-inf")).all()
