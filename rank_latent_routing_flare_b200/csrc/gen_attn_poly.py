"""Derives the polynomial of the attention kernels' FMA-pipe tanh.

tanh(u) = u p(u^2) for |u| <= 1/2, p of degree 3 with minimal maximum relative
error against tanh(sqrt(v)) / sqrt(v) on [0, 1/4] (an analytic function of v,
nearest singularity at v = -(pi / 2)^2), by the Remez exchange algorithm in
float64, rounded to float32.

Run:  python gen_attn_poly.py      (prints the coefficients and error bounds)
"""
from __future__ import annotations

import numpy as np


def tanh_ratio(v):
    v = np.asarray(v, dtype=np.float64)
    u = np.sqrt(np.maximum(v, 1e-12))
    return np.where(v < 1e-8, 1.0 - v / 3.0, np.tanh(u) / u)


def remez(f, deg: int, lo: float, hi: float, iters: int = 40):
    """Coefficients (lowest first) of the polynomial nearest to f on [lo, hi] in relative error, and that error."""
    n = deg + 2
    k = np.arange(n)
    ref = 0.5 * (lo + hi) + 0.5 * (hi - lo) * np.cos(np.pi * (n - 1 - k) / (n - 1))
    grid = np.linspace(lo, hi, 200001)
    fg = f(grid)
    c = None
    for _ in range(iters):
        A = np.zeros((n, n))
        fr = f(ref)
        for i, x in enumerate(ref):
            A[i, :deg + 1] = x ** np.arange(deg + 1)
            A[i, deg + 1] = -((-1) ** i) * fr[i]
        c = np.linalg.solve(A, fr)[:deg + 1]
        err = np.polyval(c[::-1], grid) / fg - 1.0
        segs = np.split(np.arange(grid.size), np.flatnonzero(np.diff(np.sign(err)) != 0) + 1)
        ext = np.array([s[np.argmax(np.abs(err[s]))] for s in segs])
        if len(ext) < n:
            break
        best = max(range(len(ext) - n + 1), key=lambda i: np.min(np.abs(err[ext[i:i + n]])))
        ref = grid[ext[best:best + n]]
    return c, float(np.max(np.abs(np.polyval(c[::-1], grid) / fg - 1.0)))


def tanh_coeffs():
    return remez(tanh_ratio, 3, 0.0, 0.25)


def main():
    for name, (c, e) in (("tanh", tanh_coeffs()),):
        print(f"{name}: maximum relative error {e:.3e}")
        for i, ci in enumerate(np.array(c, dtype=np.float32)):
            print(f"  c{i} = {float(ci).hex()}  ({float(ci):.9g})")


if __name__ == "__main__":
    main()
