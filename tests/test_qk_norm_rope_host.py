"""Host-only checks of the query/key preparation's entry points: refusals come
back before anything is enqueued, sizes need no GPU."""
import ctypes
import os
import re

import pytest
import torch

import rank_latent_routing_flare_b200 as fl
from rank_latent_routing_flare_b200 import Status
from rank_latent_routing_flare_b200 import qk_norm_rope as m

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "flare_ops.h")
A, W = 0x10000, 0x20000   # never dereferenced: every call fails a check, or finds no device

NAMES = ["B", "N", "D", "Hq", "Hk", "rot", "axes", "interleaved", "pos_kind", "eps", "freqs", "positions", "lengths",
         "Q", "q0", "q1", "q2", "K", "k0", "k1", "k2", "q_gain", "k_gain", "q_per_head", "k_per_head", "Qr", "r0", "r1",
         "r2", "Kr", "s0", "s1", "s2", "dQ", "t0", "t1", "t2", "dK", "u0", "u1", "u2", "dq_gain", "dk_gain"]


def args(**over):
    v = dict.fromkeys(NAMES, 0)
    v.update(B=2, N=100, D=32, Hq=4, Hk=2, rot=32, axes=1, eps=1e-6, freqs=A, Q=A, K=A, q_gain=A, k_gain=A, Qr=A,
             Kr=A, dQ=A, dK=A, dq_gain=A, dk_gain=A)
    for x, H in (("q", 4), ("r", 4), ("t", 4), ("k", 2), ("s", 2), ("u", 2)):
        v[x + "0"], v[x + "1"], v[x + "2"] = H * 100 * 32, 100 * 32, 32
    v.update(over)
    return m._ARGS.pack(*[v[n] for n in NAMES])


def fwd(**over):
    return fl.load_library().flare_qk_norm_rope_fwd(args(**over), None)


def bwd(ws=W, ws_bytes=1 << 40, **over):
    return fl.load_library().flare_qk_norm_rope_bwd(args(**over), ws, ws_bytes, None)


def test_header_is_exported_and_matches_the_packing():
    text = open(HEADER).read()
    names = set(re.findall(r"FLARE_API\s+[\w\s\*]+?\b(flare\w*)\s*\(", text))
    assert {"flare_qk_norm_rope_fwd", "flare_qk_norm_rope_bwd", "flare_qk_norm_rope_workspace_bytes"} <= names
    lib = fl.load_library()
    assert all(hasattr(lib, n) for n in names)
    body = re.search(r"typedef struct \{(.*?)\} flare_qk_norm_rope_args;", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    members = sum(3 if "[3]" in d else 1 for line in body.split(";") for d in line.split(",") if d.strip())
    assert members == len(NAMES) and m._ARGS.size == 8 * members


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(call):
    assert call(Q=0) == Status.ERR_NULL and call(Kr=0) == Status.ERR_NULL
    assert call(freqs=0) == Status.ERR_NULL
    assert call(pos_kind=1) == Status.ERR_NULL and call(positions=A) == Status.ERR_NULL
    for over in (dict(N=0), dict(B=-1), dict(Hq=-1), dict(rot=33), dict(rot=48), dict(eps=-1.0), dict(pos_kind=3),
                 dict(axes=2), dict(pos_kind=2, positions=A, axes=5), dict(rot=0), dict(q2=-32), dict(k1=8),
                 dict(Hk=0), dict(eps=float("nan"))):
        assert call(**over) == Status.ERR_SHAPE, over
    for over in (dict(D=24), dict(D=256), dict(rot=8), dict(Hq=2000), dict(N=1 << 40)):
        assert call(**over) == Status.ERR_UNSUPPORTED, over
    for over in (dict(Q=A + 8), dict(Kr=A + 2), dict(q_gain=A + 4), dict(lengths=A + 2), dict(freqs=A + 1),
                 dict(q0=12804), dict(s2=36)):
        assert call(**over) == Status.ERR_ALIGN, over


def test_backward_refusals():
    assert bwd(dQ=0) == Status.ERR_NULL
    assert bwd(q_gain=0) == Status.ERR_NULL                       # a gain's gradient without the gain
    assert bwd(ws=None) == Status.ERR_NULL
    assert bwd(ws=W + 16) == Status.ERR_ALIGN
    need = fl.flare_qk_norm_rope_workspace_bytes(2, 100, 4, 2, 32)
    assert bwd(ws_bytes=need - 256) == Status.ERR_WORKSPACE
    assert bwd(t1=0) == Status.ERR_SHAPE                           # an output row written twice
    lib = fl.load_library()
    assert lib.flare_qk_norm_rope_fwd(None, None) == Status.ERR_NULL
    assert lib.flare_qk_norm_rope_bwd(None, None, 0, None) == Status.ERR_NULL


def test_workspace_sizes():
    assert fl.flare_qk_norm_rope_workspace_bytes(1, 1, 8, 8, 16) >= 16 * 16 * 4
    assert fl.flare_qk_norm_rope_workspace_bytes(2, 8191, 32, 8, 128) % 256 == 0
    for bad in ((0, 1, 1, 1, 16), (1, 1, 0, 0, 16), (1, 1, 1, 1, 48), (1, 1, -1, 2, 16)):
        assert fl.flare_qk_norm_rope_workspace_bytes(*bad) == 0


def test_valid_calls_reach_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the pointers are not real")
    assert fwd() == Status.ERR_LAUNCH and bwd() == Status.ERR_LAUNCH
    assert fwd(Hq=0, Q=0, q_gain=0, Qr=0) == Status.ERR_LAUNCH     # keys alone
    assert fwd(rot=0, freqs=0) == Status.ERR_LAUNCH
    assert bwd(ws=None, ws_bytes=0, dq_gain=0, dk_gain=0) == Status.ERR_LAUNCH


def test_python_refusals():
    x = torch.zeros(1, 2, 3, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fl.flare_qk_norm_rope_fwd()
    with pytest.raises(TypeError):
        fl.flare_qk_norm_rope_fwd(x)                                # not on a GPU
    with pytest.raises(ValueError):
        fl.flare_qk_norm_rope_fwd(x[0])
