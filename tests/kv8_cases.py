"""Seeded cases and derived tolerances of the 8-bit KV cache tests (not collected as tests)."""
import math

import numpy as np

from oracle import kv8

# 2-norm and element bounds are not guessed: see score_error and out_error.
U24, U11, U8 = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8


def masks(kind, rows, rng):
    if kind == "causal":
        return [(1 << (r + 1)) - 1 for r in range(rows)]
    if kind == "own":
        return [1 << r for r in range(rows)]
    if kind == "none":
        return [0] * rows
    if kind == "holes":  # some rows see nothing new
        return [0 if r % 3 == 1 else int(rng.integers(0, 2 ** 63)) for r in range(rows)]
    anc = []
    for c in range(rows):
        p = int(rng.integers(0, c)) if c else -1
        anc.append((anc[p] if c else 0) | (1 << c))
    return anc


def visible(m, rows, prefix, base, n):
    vis = np.zeros((rows, n), dtype=bool)
    vis[:, :prefix] = True
    for r in range(rows):
        for e in range(rows):
            if (m[r] >> e) & 1:
                vis[r, base + e] = True
    return vis


def score_error(q, k, scale, cap):
    """Bound on |score - exact score| for q [R, Hq, hd] (fp32) and the dequantised k [n, H, hd]: [R, Hq, n].

    An fp32 q row, scaled by a power of two so that its largest magnitude is below 2^8, is hi + lo in fp16: what is
    left over is at most 2^-11 of 2^-11 of a number below 2^8, 2^-22 of twice the row's largest magnitude, for each
    element (16-bit q needs no lo and loses nothing but subnormals below 2^-24).  The products with the codes are
    exact, 128 of them are added in fp32 in at most 16 + 8 steps (a step's inner sum is at least as exact), each off
    by at most 2^-23 of the sum of magnitudes; then two fp32 roundings of the coefficient, two of the product (and
    tanh's few, whose error the cap multiplies: 4 2^-23 of the cap)."""
    group = q.shape[1] // k.shape[1]
    kk = np.repeat(np.abs(k.astype(np.float64)), group, 1)
    aq = np.abs(q.astype(np.float64))
    rest = 2.0 ** -21 * aq.max(-1)[..., None] * kk.sum(-1).T[None]
    mags = np.matmul(aq.transpose(1, 0, 2), kk.transpose(1, 2, 0)).transpose(1, 0, 2)
    return scale * (rest + 24 * 2.0 ** -23 * mags + 4 * U24 * mags) + (8 * 2.0 ** -23 * cap if cap else 0.0)


def out_error(q, k, v, vis, want, scale, cap, io):
    """Bound on |out - exact out|.  A softmax weight p is off by its score's error e (and the maximum's), by the
    exponential's 2^-22 and, relative to the largest weight 1, by its rounding: 2^-22 (hi + lo) for fp32, 2^-11 of
    itself (one fp16) for 16-bit types; then sums of n terms in fp32 in at most n / 16 + 200 steps."""
    n = vis.sum(1)[:, None].astype(np.float64)
    e = np.where(vis[:, None, :], score_error(q, k, scale, cap), 0.0).max(-1)
    group = q.shape[1] // k.shape[1]
    vv = np.repeat(np.abs(v.astype(np.float64)), group, 1)
    s = np.where(vis[:, None, :], kv8.scores(q, k, scale, cap), -np.inf)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    total = np.maximum(p.sum(-1), 1e-300)
    seen = np.where(vis.any(0)[:, None, None], vv, 0.0)
    mean_v = np.matmul(p.transpose(1, 0, 2), seen.transpose(1, 0, 2)).transpose(1, 0, 2) / total[..., None]
    top = np.where(vis.any(0)[:, None, None], vv, 0.0).max((0, 2))[None, :]
    rel = 2 * (2 * e + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(m[..., 0]), m[..., 0], 0.0)))) + (n / 16 + 200) * 2.0 ** -23
    rel = rel + (2.0 ** -21 if io == "fp32" else 2.0 ** -11)
    # weights that end below fp16's smallest step: 2^-24 under 2^9 (the tensor-core kernel; 2^14 elsewhere), half of it
    floor = n * 2.0 ** -34 * top / total
    out = rel[..., None] * mean_v + floor[..., None]
    half = {"fp32": U24, "bf16": U8, "fp16": U11}[io]
    # fp16 numbers below 2^-14 lie 2^-24 apart: rounding to one is off by up to 2^-25 whatever the value (an output of
    # 2.4e-6 was off by 2.8e-8 = 0.93 of that, 2^-11 of the value being 1.1e-9)
    return out + half * (np.abs(want) + out) + (2.0 ** -25 if io == "fp16" else 1e-30)


def lse_error(q, k, vis, lse, scale, cap):
    """Bound on |lse - exact lse|: the scores' error, the sum's and the logarithm's roundings."""
    e = np.where(vis[:, None, :], score_error(q, k, scale, cap), 0.0).max(-1)
    n = vis.sum(1)[:, None]
    a = np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return e + (n / 8 + 200) * U24 + 8 * U24 * (a + 16)


def make_rows(rng, n, heads, hd, io):
    """K-like rows with a few large channels, rounded to the io type; fp32 array."""
    import torch

    x = rng.standard_normal((n, heads, hd)) * (0.5 + rng.random((n, heads, 1)))
    x[..., :: max(1, hd // 4)] *= 6.0
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[io]
    return torch.tensor(x, dtype=torch.float32).to(dt)
