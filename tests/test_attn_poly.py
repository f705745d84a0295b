"""The FMA-pipe tanh of the attention kernels (ScoreOps in csrc/attn_math.cuh),
emulated in IEEE fp32 on the CPU: its constants are the ones gen_attn_poly.py
derives, and capped scores stay within the polynomial's error."""
import importlib.util
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_latent_routing_flare_b200", "csrc")


def kernel_coeffs():
    text = open(os.path.join(CSRC, "attn_math.cuh")).read()
    return np.array([float.fromhex(h) for h in re.findall(r"f2_dup\((-?0x1\.[0-9a-f]+p-?\d+)f \* f", text)], dtype=np.float32)


def generator():
    spec = importlib.util.spec_from_file_location("gen_attn_poly", os.path.join(CSRC, "gen_attn_poly.py"))
    gen = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(gen)
    return gen


def test_constants_come_from_the_generator():
    c, err = generator().tanh_coeffs()
    assert len(kernel_coeffs()) == 4 and np.array_equal(kernel_coeffs(), np.array(c, dtype=np.float32))
    assert err < 6e-7


def f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32)


@pytest.mark.parametrize("scale,cap", [(0.25, 30.0), (1.0, 1.0), (1.0, 5e4), (0.088, 50.0), (3.0, 0.02)])
def test_capped_scores(scale, cap):
    """cap log2(e) tanh(s scale / cap) for |s scale / cap| <= 1/2: the polynomial's 5.5e-7 and four fp32 products
    (the coefficients) and four fused steps, each half a step of 2^-23, relative."""
    c = kernel_coeffs()
    u, out = np.float32(scale) / np.float32(cap), np.float32(cap) * np.float32(1.4426950408889634)
    f, w2 = f32(np.float64(u) * out), f32(np.float64(u) * u)
    k = [f32(np.float64(c[0]) * f), None, None, None]
    p = f32(np.float64(f) * w2)
    for i in (1, 2, 3):
        k[i] = f32(np.float64(c[i]) * p)
        p = f32(np.float64(p) * w2)
    s = f32(np.linspace(-0.5, 0.5, 100001) / np.float64(u))
    w = f32(s.astype(np.float64) ** 2)
    acc = k[3]
    for i in (2, 1, 0):
        acc = f32(acc.astype(np.float64) * w + k[i])
    got = f32(s.astype(np.float64) * acc).astype(np.float64)
    want = cap * np.log2(np.e) * np.tanh(s.astype(np.float64) * scale / cap)
    assert np.all(np.abs(got - want) <= (5.5e-7 + 12 * 2.0 ** -24) * np.abs(want))
