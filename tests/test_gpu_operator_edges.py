"""Calls at the edges of what the attention and the preparation of queries and
keys allow: caps so large that they hardly bend a score, long packed
sequences, other streams, captured autograd, two calls at once."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import rank_latent_routing_flare_b200 as fl

from . import attention_ref as ref
from .test_gpu_attention import DEV, check, i32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [16, 128])
@pytest.mark.parametrize("cap", [1e4, 1e6, 1e9])
@pytest.mark.parametrize("bias", [False, True])
def test_a_huge_cap_leaves_scores_alone(D, cap, bias):
    """cap tanh(s / cap) = s (1 - (s / cap)^2 / 3 + ..): below 2e-7 s for scores up to 7 under these caps.  The bound is
    the one without a cap, whose share for the scores' roundings, (D + 8) 2^-24 times the sum of |q| |k|, is some ten
    times that and the polynomial's 5.5e-7 together."""
    for Nq in (1, 150):
        Q, K, V, dY, o = make(1, 2, 1, Nq, 300, D, seed=D, bias=bias)
        want = ref.attention(Q, K, V, dY=dY, **o)
        Y, L = fl.flare_attention_fwd_train(Q, K, V, cap=cap, **o)
        ref.close(Y, want["Y"], "Y")
        ref.close(L, want["L"], "L")
        for name, got in zip(("dQ", "dK", "dV"), fl.flare_attention_bwd(Q, K, V, Y, L, dY, cap=cap, **o)):
            ref.close(got, want[name], name)


@pytest.mark.parametrize("cap", [1e-6, 1e-3, 0.05])
def test_a_tiny_cap(cap):
    """Scores of almost nothing: every weight is about 1 / n, every gradient of Q and K is the cap's derivative."""
    for Nq in (2, 150):
        check(*make(2, 2, 1, Nq, 200, 64, seed=21, cap=cap, causal=True, lengths=i32(200, 77)), backward=Nq > 2)


@pytest.mark.parametrize("cap", [30.0, 55.0, 56.0, 90.0])
def test_hidden_scores_far_above_the_visible(cap):
    """The keys behind a row score near half the cap, the ones it sees near minus half of it; some hidden keys are
    NaN or infinite.  On either side of the cap up to which hidden columns count for a tile's reference."""
    g = torch.Generator(device=DEV).manual_seed(31)
    for D in (16, 64, 128):
        N, edge = 500, 250
        Q = torch.full((1, 2, N, D), 1.0, device=DEV).bfloat16()
        K = torch.randn(1, 2, N, D, generator=g, device=DEV) * 0.1
        K[:, :, :edge] -= 0.45 * cap / D ** 0.5
        K[:, :, edge:] += 0.45 * cap / D ** 0.5
        V = torch.randn(1, 2, N, D, generator=g, device=DEV).bfloat16()
        o = {"cap": cap, "prefix": i32(edge), "causal": True, "q_offsets": i32(-1000)}
        check(Q, K.bfloat16(), V, torch.randn(1, 2, N, D, generator=g, device=DEV).bfloat16(), o)
        ids = torch.zeros(1, N, dtype=torch.int32, device=DEV)
        ids[:, edge:] = -1                                       # check puts NaN and infinities there
        o = {"cap": cap, "documents": ids}
        check(Q, K.bfloat16(), V, torch.randn(1, 2, N, D, generator=g, device=DEV).bfloat16(), o)


@pytest.mark.parametrize("slope", [-0.05, 0.0, 3.0])
def test_slopes_of_any_sign(slope):
    """A negative slope prefers distant keys; a zero one is no bias."""
    for Nq in (2, 300):
        Q, K, V, dY, _ = make(1, 2, 1, Nq, 700, 32, seed=22)
        o = {"slopes": torch.tensor([slope, -slope / 2], device=DEV)}
        check(Q, K, V, dY, dict(o), backward=Nq > 2)
        check(Q, K, V, dY, dict(o, causal=True, cap=9.0), backward=Nq > 2)


@pytest.mark.parametrize("N,cuts,dead", [
    (16 * 1024, (), ()), (16 * 1024, (1024, 15 * 1024), (1,)),                        # one launch
    (17 * 1024, (), ()), (33 * 1024, (5, 1023, 1024, 20000, 32767, 32768), (4,)),  # in three
    (40001, (40000,), ()), (70000, (1, 2, 3, 65535, 65536, 65537, 69999), (1, 6))])
def test_documents_of_long_sequences(N, cuts, dead):
    g = torch.Generator(device=DEV).manual_seed(23)
    where = sorted({0, N - 3} | {max(0, min(N - 3, c - 1)) for c in cuts} | {1022, N // 2})
    B = len(where)
    ids = torch.zeros(N, dtype=torch.int32)
    for n, c in enumerate(cuts):
        ids[c:] = -1 if n + 1 in dead else n % 2 + 1
    for Nq in (3, 20):
        Q = torch.randn(B, 1, Nq, 16, generator=g, device=DEV).bfloat16()
        K, V = (torch.randn(B, 1, N, 16, generator=g, device=DEV).bfloat16() for _ in range(2))
        o = {"documents": ids.expand(B, N).contiguous().to(DEV), "q_offsets": i32(*where)}
        check(Q, K, V, Q.clone(), o, backward=False)


def test_memory_of_a_call_on_another_stream_is_not_handed_out_early():
    """What a call allocates for itself stays its own until its stream has got there."""
    Q, K, V, _, _ = make(1, 2, 2, 1, 40000, 64, seed=24)                 # splits joined through the workspace
    x = torch.randn(2, 3000, 4 * 32, device=DEV).bfloat16().unflatten(-1, (-1, 32)).transpose(1, 2)
    dy, gain = torch.randn_like(x, memory_format=torch.contiguous_format), torch.ones(32, device=DEV)
    want = fl.flare_attention_fwd(Q, K, V)
    wantg = fl.flare_qk_norm_rope_bwd(x, None, dy, None, gain)
    size = [fl.flare_attention_workspace_bytes(1, 2, 2, 1, 40000, 64), fl.flare_qk_norm_rope_workspace_bytes(2, 3000, 4, 0, 32)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                                    # some 10 ms
    Y = fl.flare_attention_fwd(Q, K, V, stream=side)
    g = fl.flare_qk_norm_rope_bwd(x, None, dy, None, gain, stream=side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        mine = torch.cuda.Event()
        mine.record()
    junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in size for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and torch.equal(g["dq_gain"], wantg["dq_gain"]) and torch.equal(g["dQ"], wantg["dQ"])
    assert all((j == 255).all() for j in junk)


def test_captured_autograd():
    """Forward and backward of both operators in one graph, replayed on other inputs."""
    B, N, Hq, Hk, D = 2, 150, 4, 2, 32
    gen = torch.Generator(device=DEV).manual_seed(25)
    packed = torch.randn(B, N, (Hq + 2 * Hk) * D, generator=gen, device=DEV).bfloat16().requires_grad_()
    gain = torch.ones(D, device=DEV).requires_grad_()
    freqs = 10000.0 ** (-torch.arange(D // 2, device=DEV) / (D // 2))
    dY = torch.randn(B, Hq, N, D, generator=gen, device=DEV).bfloat16()

    def step():
        rows = packed.unflatten(-1, (-1, D)).transpose(1, 2)
        Qr, Kr = fl.flare_qk_norm_rope(rows[:, :Hq], rows[:, Hq:Hq + Hk], gain, gain, freqs)
        Y = fl.flare_attention(Qr, Kr, rows[:, Hq + Hk:], causal=True, cap=20.0)
        return (Y, *torch.autograd.grad(Y, (packed, gain), dY))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        packed.mul_(0.7)
        gain.add_(0.3)
    want = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_no_second_derivatives():
    x = torch.randn(1, 2, 9, 16, device=DEV).bfloat16().requires_grad_()
    for y in (fl.flare_attention(x, x, x), fl.flare_qk_norm_rope(x, None)[0]):
        (g,) = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.float().sum().backward()


def test_one_tensor_as_query_key_and_value():
    x = torch.randn(2, 2, 130, 32, device=DEV).bfloat16()
    check(x.clone(), x.clone(), x.clone(), torch.randn_like(x), {"causal": True})
    same = fl.flare_attention_fwd(x, x, x, causal=True)
    assert torch.equal(same, fl.flare_attention_fwd(x.clone(), x.clone(), x.clone(), causal=True))


def test_two_threads_and_two_streams_at_once():
    """Calls that run at the same time, each with its own workspace, do not see one another."""
    jobs = [make(1, 2, 1, 1, 30000, 64, seed=26), make(2, 4, 2, 300, 300, 64, seed=27, causal=True, cap=5.0),
            make(1, 8, 1, 200, 500, 32, seed=28, bias=True)]
    want = [fl.flare_attention_fwd_train(*j[:3], **j[4]) for j in jobs]
    grads = [fl.flare_attention_bwd(*j[:3], *w, j[3], **j[4]) for j, w in zip(jobs, want)]
    torch.cuda.synchronize()
    bad = []

    def run(j, w, gw):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                Y, L = fl.flare_attention_fwd_train(*j[:3], **j[4])
                g = fl.flare_attention_bwd(*j[:3], Y, L, j[3], **j[4])
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(Y, w[0]) and torch.equal(L, w[1]) and all(torch.equal(a, b) for a, b in zip(g, gw))):
                    bad.append(j[0].shape)

    threads = [threading.Thread(target=run, args=a) for a in zip(jobs, want, grads)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_preparation_of_many_heads_and_single_rows():
    """As many heads as a call takes, and one row of one head, against the same rows prepared on their own."""
    gen = torch.Generator(device=DEV).manual_seed(29)
    x = torch.randn(1, 250, 5, 128, generator=gen, device=DEV).bfloat16()
    gains = 1 + 0.1 * torch.randn(250, 128, generator=gen, device=DEV)
    freqs = 10000.0 ** (-torch.arange(64, device=DEV) / 64)
    y, _ = fl.flare_qk_norm_rope_fwd(x, None, gains, freqs=freqs)
    for h in (0, 100, 249):
        one, _ = fl.flare_qk_norm_rope_fwd(x[:, h:h + 1], None, gains[h].clone(), freqs=freqs)
        assert torch.equal(one, y[:, h:h + 1])
    last, _ = fl.flare_qk_norm_rope_fwd(x[:, 7:8, 4:5], None, gains[7].clone(), freqs=freqs, positions=i32(4).view(1, 1))
    assert torch.equal(last, y[:, 7:8, 4:5])


def test_offsets_beyond_32_bits():
    """Batch entries 2^31 elements apart, in every tensor that takes strides."""
    far, N, D = 1 << 31, 150, 32
    whole = torch.empty(far + 4 * N * D, dtype=torch.bfloat16, device=DEV)

    def rows(n):   # the n-th tensor of two batch entries and one head
        return whole.as_strided((2, 1, N, D), (far, N * D, D, 1), n * N * D)

    Q, K, V, dY, _ = make(2, 1, 1, N, N, D, seed=30)
    want = fl.flare_attention_fwd_train(Q, K, V, causal=True)
    grads = fl.flare_attention_bwd(Q, K, V, *want, dY, causal=True)
    for n, t in enumerate((Q, K, V)):
        rows(n).copy_(t)
    Y, L = fl.flare_attention_fwd_train(rows(0), rows(1), rows(2), Y=rows(3), causal=True)
    assert torch.equal(Y, want[0]) and torch.equal(L, want[1])
    step = fl.flare_attention_fwd(rows(0)[:, :, -1:], rows(1), rows(2), causal=True)
    assert torch.equal(step, fl.flare_attention_fwd(Q[:, :, -1:], K, V, causal=True))
    got = fl.flare_attention_bwd(rows(0), rows(1), rows(2), Y, L, dY, causal=True, dV=rows(3))
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    freqs = 100.0 ** (-torch.arange(D // 2, device=DEV) / (D // 2))
    Qr, Kr = fl.flare_qk_norm_rope_fwd(Q, K, freqs=freqs)
    got = fl.flare_qk_norm_rope_fwd(rows(0), rows(1), freqs=freqs, Qr=rows(2), Kr=rows(3))
    assert torch.equal(got[0], Qr) and torch.equal(got[1], Kr)
    back = fl.flare_qk_norm_rope_bwd(Q, K, Qr, Kr, freqs=freqs)
    got = fl.flare_qk_norm_rope_bwd(rows(0), rows(1), rows(2), rows(3), freqs=freqs)
    assert torch.equal(got["dQ"], back["dQ"]) and torch.equal(got["dK"], back["dK"])


FIRST = """
import torch, rank_latent_routing_flare_b200 as fl
Q, K, V = (torch.randn(1, 4, 300, 64, device='cuda').bfloat16() for _ in range(3))
gain, freqs = torch.ones(64, device='cuda'), torch.rand(32, device='cuda')
ids = torch.zeros(1, 300, dtype=torch.int32, device='cuda')
def step():
    leaves = [t.detach().requires_grad_() for t in (Q, K, V)]
    Qr, Kr = fl.flare_qk_norm_rope(leaves[0], leaves[1], gain, gain, freqs)
    Y = fl.flare_attention(Qr, Kr, leaves[2], documents=ids, causal=True)
    return (Y, fl.flare_attention_fwd(Q[:, :, -1:], K, V), *torch.autograd.grad(Y, leaves, V))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, want))
print('same')
"""


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing has been loaded, and the backward's thread has no context yet, when the capture begins."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
